// lr_heads_tensor.cu -- selective scan with heads, bf16 I/O, on the sm_103a tensor
// cores (tcgen05, accumulators in TMEM, operands by TMA):
//
//   S_t = a_t S_{t-1} + d_t x_t B_t^T,   y_t = (S_t C_t + skip x_t) silu(z_t),
//   d_t = softplus(dt_t + bias),   a_t = exp(-exp(A_log) d_t)
//
// The chunked form is the decayed attention's (lr_decay_tensor.cu, whose comment has the
// mathematics, the precision and what infinities do), with q = C, k = B, v = x and a
// step size beside every decay weight:
//
//   O  = [(Q K^T) . D] V + diag(2^L) Q S^T + skip V,   D_ts = d_s 2^(L_t - L_s), s <= t
//   S' = 2^L_C S + sum_s d_s 2^(L_C - L_s) v_s k_s^T
//
// The step sizes go into the factors that the columns of Q K^T and the state's weights
// have anyway.  The skip is added by the output warps in fp32 (on the diagonal of Q K^T,
// which is rounded to bf16, it would lose its own last bits); they take their part of V
// into registers before they wait for the chunk's products, so that they hold its tile no
// longer than the products do.
//
// What the gates come to is made by a launch of its own: softplus, the sums of log
// decays in 64-bit fixed point and the powers are the same for every block of a head's
// value rows, and one warp of the main kernel that did them took longer than a chunk
// (10000 clocks of a chunk's 4600 with the library's log1pf, 4200 without a softplus).
// Per step it leaves the state's weight, the readout's factor and the step's own two
// values, per chunk the column factors, and each role of the main kernel loads its own
// a chunk ahead.
//
// A steep chunk (past 2^-40) forms D in blocks of 16 columns: rows past the block take it
// as 2^(L_t - L_e) times the columns' d_s 2^(L_e - L_s), e the block's last step, both
// <= 1; only the two blocks that a row's diagonal crosses take a power an element.
//
// A thread block owns 64 value rows of one (batch row, head, time segment), 128 key
// columns.  Roles, connected by mbarriers: state (8 warps), output (8: 32 rows by 32
// columns a warp), front (8), weight (4), TMA, and one warp for each of dS, P and O's
// products.  TMEM: P 2 x 128 columns (PD inside), O 2 x 64, so that the gate and the stores
// of one chunk's outputs stand in no chunk's way, dS 2 x 64, onto which the three terms of
// the state's weights add up (side by side, as in the decayed attention, they would take
// the columns of O's second buffer).
//
// Measured (bf16 H16 P128 N128, back to back in a graph): B4 L4096 with skip and gate 117.7
// us, which is 1.8 TB/s of its 214 MB and 145 TFLOP/s; without the gate 99.5, without the
// skip 108; every chunk steep 121; B1 L32768 308, without the gate 264, 4 segments (gates
// 20, the segments' states 70, the rest outputs); B8 L1017 H32 P64 N64 69.7.  The chunk is
// a chain of hand-overs between the roles, with one block on 128 of 152 SMs: issue 38 %,
// tensor pipe 22 %, LSU 40 %, DRAM 26 %.
//   adopted, each against the one before (B4 L4096 with gate, us): gates by a launch of their
//   own 222 -> 146; outputs through P's free columns, stores by whole sectors 130; work
//   shared evenly over the schedulers, fewer operations 124.6; the gate's tile by TMA and two
//   accumulators of outputs 112; whole quarters of weights without a gate 109.6; the skip in
//   fp32 instead of on the bf16 diagonal 118.5, the gate's tile handed back earlier 117.7
//   rejected: z a chunk ahead in registers 149 to 153 (spills); the weights' loop unrolled
//   twice 112, four times 125 (the roles share an instruction cache); two or four buffers of
//   column factors, a suspend time in the waits, the gates' launch in clusters of four: no
//   change.  Of the skip: into the accumulator ahead of the products, by the output warps 135
//   (it waits for the next V), by the front warps 125; x read once the products are there 120,
//   from global memory 137; the gate's tile taken early too 132 to 139 (registers); the next
//   tiles of V and of the gate prefetched into L2 117.5; on the diagonal in two bf16 terms 116,
//   16 bits
#include "lr_decay_tensor.cuh"

namespace lr {

namespace ht {
using dt::arrive;
using dt::Ctl;
using dt::elect_one;
using dt::hi_f;
using dt::kRescaleTensor;
using dt::kSteepChunk;
using dt::lo_f;
using dt::not_finite;
using dt::pack;
using dt::three_terms;
using dt::wait_slow;
constexpr int C = kDecayChunk;
constexpr int RB = kDecayRows;
// State warps 0 .. 7, output 8 .. 15, then front and weight.  A warp reaches the TMEM rows of
// its number modulo 4, which is also the scheduler that it runs on, and rows 32 w .. of P
// have 2 w + 2 blocks of columns under the diagonal: one front warp for the first rows,
// two, two and three for the others, and the weight warps where there are fewer of them.
constexpr int OUT = 8, FRONT = 16, TMA_WARP = 28, DS_WARP = 29, P_WARP = 30;   // 31: O
__device__ __forceinline__ bool is_weight(int warp) { return warp == 20 || (warp >= 24 && warp < 27); }
constexpr int THREADS = 32 * 32;

// What the gates' launch leaves of a chunk.
struct Chunk {
    float col[C];    // column factors of P: w d; steep: d 2^(L_e - L_s), e the last step of s' 16
    float m;         // the state's factor (1: none)
    int steep;
    long long total; // the chunk's log2 decay
    int last[8];     // steep: L of every 16 steps' last, see units_of
    float after;     // the decay of the segment's chunks after it (segments but the last)
    int pad[3];
};
static_assert(sizeof(Chunk) == kChunkRecord, "");

constexpr uint32_t HALF = C * 128;              // 64 columns of Q or K: 128 rows of 128 bytes
constexpr uint32_t Q_BYTES = 2 * HALF, V_BYTES = C * RB * 2;
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * Q_BYTES, OFF_V = 4 * Q_BYTES;
constexpr uint32_t OFF_SB = OFF_V + 2 * V_BYTES;    // bf16 state [128 j][64 i]
// The state's weighted values, three terms of [4 quarters][32 s][64 i].  With a gate half of a
// quarter's steps at a time, and its tile [128 s][64 i] in the room that this leaves (without
// a gate that costs 90 -> 103 us at B4 L4096 H16 P128 N128).
template <bool GATE>
struct Weights {
    static constexpr int HALVES = GATE ? 2 : 1, STEPS = 32 / HALVES, GROUPS = 8 / HALVES;
    static constexpr uint32_t TERM = 4 * STEPS * RB * 2;
};
constexpr uint32_t OFF_W = OFF_SB + 128 * RB * 2, OFF_Z = OFF_W + 3 * Weights<true>::TERM;
constexpr uint32_t OFF_G = OFF_W + 3 * Weights<false>::TERM;   // 2 x Chunk
static_assert(OFF_Z + V_BYTES <= OFF_G, "the gate's tile");
constexpr uint32_t OFF_BAR = OFF_G + 2 * kChunkRecord;
// barriers; [2] by chunk parity, [4] by quarter
enum {
    FULL_Q = 0, EMPTY_Q = 2, FULL_K = 4, EMPTY_K = 6, FULL_V = 8, EMPTY_V = 10,
    FULL_G = 12,     // the chunk's record
    P_READY = 14,    // P_c complete
    F_DONE = 16,     // PD_c written (8 front warps)
    K_DONE = 18,     // chunk c's accumulator read (8 output warps)
    OX_DONE = 20,    // Q S^T complete: the bf16 state has been read
    O_DONE = 22,
    W_READY = 24,    // weighted values of a quarter, or of half of it, twice a chunk
    W_FREE = 28,
    DS_DONE = 32, DS_FREE = 34,   // [2]
    FULL_Z = 36, EMPTY_Z,
    SB_READY,        // bf16 state before chunk c (8 state warps)
    FIX,             // a steep chunk's Q S^T scaled (8 output warps)
    MMA_END, NBAR
};
constexpr uint32_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr uint32_t OFF_CTL = OFF_TMEM + 8;
constexpr uint32_t SMEM = OFF_CTL + 40;
static_assert(OFF_BAR % 8 == 0 && OFF_CTL % 8 == 0, "");
static_assert(SMEM <= 227 * 1024, "one block per SM");

constexpr uint32_t T_P = 0, T_O = 256, T_DS = 384;   // 2 x 128, 2 x 64, 2 x 64 columns
constexpr uint32_t IDESC_P = umma_idesc_bf16(128, 128, 0, 0);
constexpr uint32_t IDESC_O = umma_idesc_bf16(128, 64, 0, 1);
constexpr uint32_t IDESC_DS = umma_idesc_bf16(128, 64, 1, 1);

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// 16 bytes of shared memory, read here: a plain load whose value only some lanes come to use
// was moved down to them, past the hand-over of what it reads.
__device__ __forceinline__ uint4 read_now(const void *p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(smem_u32(p))
                 : "memory");
    return v;
}

// The neighbouring lane's value.
__device__ __forceinline__ uint4 xor1(uint4 v) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, 1), __shfl_xor_sync(0xffffffffu, v.y, 1),
                      __shfl_xor_sync(0xffffffffu, v.z, 1), __shfl_xor_sync(0xffffffffu, v.w, 1));
}

// Position of a (batch row, head)'s step in the gates' arrays, and of its chunk's record.
__device__ __forceinline__ size_t step_at(const DecayArgs &a, int64_t bh, int64_t t) {
    return size_t(bh) * ((a.L + C - 1) / C * C) + t;
}
__device__ __forceinline__ const unsigned char *record_at(const DecayArgs &a, int64_t bh, int64_t t) {
    return a.hd.chunk + step_at(a, bh, t) / C * kChunkRecord;
}
}  // namespace ht

// ---------------------------------------------------------------------------
// The gates.  A block takes one (batch row, head, segment), a warp one chunk at a time
// (lane i: steps 4 i .. 4 i + 3), as many chunks at once as it has warps: sums within
// the chunk, then, from the chunks' totals, which warp 0 goes through, whether the state
// is rescaled at each and what decay has been left before it.  (Every warp going through
// them: 15.7 us under a profiler at B4 L4096 H16, most of that issue slots; so 12.5, of which
// the loads of dt, H elements apart, are most.  In clusters of four blocks: no change behind
// the call.)
__global__ void __launch_bounds__(1024) heads_gates_kernel(const __grid_constant__ DecayArgs a, StatusRef sref) {
    using namespace ht;
    using bf = __nv_bfloat16;
    __shared__ long long totals[32], before_of[32];
    __shared__ int how_of[32];   // bit 0: rescaled, bit 1: steep
    // the main kernel reads the call's inputs as soon as it runs, so it may start only
    // once the kernel before this one has ended
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (threadIdx.x == 0 && blockIdx.x == 0) status_begin(sref);
    const int seg = blockIdx.x % a.n_seg;
    const int64_t bh = blockIdx.x / a.n_seg;
    const int h = int(bh % a.H), b = int(bh / a.H);
    const int64_t s0 = int64_t(seg) * a.seg_len;
    const int nrun = int(max(int64_t(0), min(int64_t(dec::row_len(a.lens, b, a.L)), min(a.L, s0 + a.seg_len)) - s0));
    const int n_chunks = (nrun + C - 1) / C;
    const dec::Gates<true> gates(a, h);
    const bf *g = static_cast<const bf *>(a.g) + (size_t(b) * a.L + s0) * a.hd.ldg + h;
    auto record_of = [&](int c) {
        return reinterpret_cast<Chunk *>(const_cast<unsigned char *>(record_at(a, bh, s0 + int64_t(c) * C)));
    };
    bool bad = false;
    long long base = 0, tot = 0;
    // steps 4 lane .. of chunk c: step sizes and decays since the chunk's start
    float delta[4];
    long long l[4], all;
    auto chunk = [&](int c) {
        float gv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = c * C + 4 * lane + i;
            gv[i] = t < nrun ? __bfloat162float(g[size_t(t) * a.hd.ldg]) : 0.0f;
        }
        long long run = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float ld = gates.of(gv[i], delta[i]);
            if (c * C + 4 * lane + i < nrun)
                run += dec::to_fix(ld, bad);
            else
                delta[i] = 0.0f;
            l[i] = run;
        }
        long long incl = run;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, m);
            if (lane >= m) incl += up;
        }
        all = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] += incl - run;
    };
    for (int c0 = 0; c0 < n_chunks; c0 += warps) {
        const int c = c0 + warp;
        all = 0;
        if (c < n_chunks) chunk(c);
        if (lane == 0) totals[warp] = all;
        __syncthreads();
        if (warp == 0) {   // (it alone holds base and tot)
            const int n = min(warps, n_chunks - c0);
            const long long mine = lane < n ? totals[lane] : 0;
            const uint32_t steep_of = __ballot_sync(0xffffffffu, mine < kSteepChunk);
            long long kept = 0;
            uint32_t re_of = 0;
            static_assert((kRescaleTensor & 0xffffffffll) == 0, "a comparison of the upper halves");
#pragma unroll 8
            for (int j = 0; j < n; ++j) {   // few operations: one warp, and each needs the last
                if (j == lane) kept = base;
                base += __shfl_sync(0xffffffffu, mine, j);
                if ((steep_of >> j & 1) != 0 || int(base >> 32) < int(kRescaleTensor >> 32)) base = 0, re_of |= 1u << j;
            }
            before_of[lane] = kept;
            how_of[lane] = int(re_of >> lane & 1) + 2 * int(steep_of >> lane & 1);
            long long sum = mine;
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            tot = max(tot + sum, -(1ll << 60));
        }
        __syncthreads();
        const long long before = before_of[warp], end = before + all;
        const bool re = how_of[warp] & 1, steep = how_of[warp] & 2;
        if (c >= n_chunks) continue;
        float w[4], r[4], col[4];
        int u[4];
        const long long last = __shfl_sync(0xffffffffu, l[3], lane | 3);   // of the lane's 16 steps
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long e = re ? all - l[i] : -(before + l[i]);
            const float p = dec::exp2_fix(e);
            w[i] = p * delta[i];
            u[i] = dec::units_of(l[i]);
            if (steep) {
                r[i] = -dec::exp2_fix(before + l[i]);   // (its sign says so, -0 too)
                col[i] = delta[i] * dec::exp2_fix(last - l[i]);
            } else {
                r[i] = dec::exp2_fix(-e);
                col[i] = w[i];
            }
        }
        const size_t at = step_at(a, bh, s0 + int64_t(c) * C + 4 * lane);
        *reinterpret_cast<float4 *>(a.hd.weight + at) = make_float4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<float4 *>(a.hd.readout + at) = make_float4(r[0], r[1], r[2], r[3]);
        float4 *own = reinterpret_cast<float4 *>(a.hd.own + at);
        own[0] = make_float4(delta[0], __int_as_float(u[0]), delta[1], __int_as_float(u[1]));
        own[1] = make_float4(delta[2], __int_as_float(u[2]), delta[3], __int_as_float(u[3]));
        if (seg < a.n_seg - 1) {   // weights to the chunk's end, for the state that the segment leaves
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = delta[i] * dec::exp2_fix(all - l[i]);
            *reinterpret_cast<float4 *>(a.hd.to_end + at) = make_float4(e[0], e[1], e[2], e[3]);
        }
        Chunk *rec = record_of(c);
        reinterpret_cast<float4 *>(rec->col)[lane] = make_float4(col[0], col[1], col[2], col[3]);
        if ((lane & 3) == 3) rec->last[lane >> 2] = u[3];
        if (lane == 0) rec->m = re ? dec::exp2_fix(end) : 1.0f, rec->steep = steep, rec->total = all;
    }
    // the decay that the scaled state still lacks when the segment is done
    if (threadIdx.x == 0) a.hd.left[bh * a.n_seg + seg] = dec::exp2_fix(base);
    if (seg < a.n_seg - 1) {   // what decays after each chunk, from the last one back
        __syncthreads();       // the records
        if (warp == 0) {
            if (lane == 0) a.seg_tot[bh * (a.n_seg - 1) + seg] = tot;
            long long after = 0;
            for (int c1 = n_chunks; c1 > 0; c1 -= 32) {
                const int c = c1 - 1 - lane;
                Chunk *rec = c >= 0 ? record_of(c) : nullptr;
                const long long t = c >= 0 ? rec->total : 0;
                long long incl = t;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const long long up = __shfl_up_sync(0xffffffffu, incl, m);
                    if (lane >= m) incl += up;
                }
                if (c >= 0) rec->after = dec::exp2_fix(after + incl - t);
                after = max(after + __shfl_sync(0xffffffffu, incl, 31), -(1ll << 60));
            }
        }
    }
    if (bad) status_report(sref, LR_ERR_RANGE);
}

// ---------------------------------------------------------------------------
// The state that a segment builds from its own steps (segmented calls): the decayed
// attention's kernel of this kind (lr_decay_tensor.cu), with the weights to the
// segment's end from the gates' launch.
namespace hs {
constexpr int C = kDecayChunk, RB = kDecayRows;
constexpr int NS = 3, NW = 3;
constexpr int WEIGHTS = 8, TMA_WARP = 8, MMA_WARP = 9, THREADS = 10 * 32;
constexpr uint32_t HALF = C * 128, K_BYTES = 2 * HALF, V_BYTES = C * RB * 2;
constexpr uint32_t T_BYTES = 64 * RB * 2;      // one term of half a chunk
constexpr uint32_t OFF_K = 0, OFF_V = NS * K_BYTES, OFF_W = OFF_V + NS * V_BYTES;
constexpr uint32_t OFF_BAR = OFF_W + NW * 3 * T_BYTES;
enum {
    FULL_K = 0, EMPTY_K = FULL_K + NS, FULL_V = EMPTY_K + NS, EMPTY_V = FULL_V + NS,
    W_READY = EMPTY_V + NS, W_FREE = W_READY + NW, DONE = W_FREE + NW, NBAR
};
constexpr uint32_t OFF_CTL = OFF_BAR + NBAR * 8;
constexpr uint32_t OFF_TMEM = OFF_CTL + 40;
constexpr uint32_t SMEM = OFF_TMEM + 8;
static_assert(SMEM <= 227 * 1024, "one block per SM");
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t IDESC = umma_idesc_bf16(128, 192, 1, 1);
}  // namespace hs

template <bool PARTS>
__global__ void __launch_bounds__(hs::THREADS, 1)
    heads_state_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ DecayArgs a, int n_vt, uint64_t timeout_ns, StatusRef sref) {
    using namespace hs;
    using dt::arrive;
    using dt::Ctl;
    using dt::hi_f;
    using dt::lo_f;
    using dt::pack;
    using bf = __nv_bfloat16;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the gates.  The main launch's first segments read them too, and wait for nothing
    // else, so it may start only once they are there
    grid_dependency_wait();
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
    const int b = dec::row_at(a, x / a.H, reinterpret_cast<int *>(sm + OFF_W)), bh = b * a.H + h;
    const int len = dec::row_len(a.lens, b, a.L);
    const int s0 = int(int64_t(seg) * a.seg_len);
    const int nrun = max(0, min(len, int(min(a.L, int64_t(s0) + a.seg_len))) - s0);
    const int n_chunks = (nrun + C - 1) / C;
    // the block's key columns: k0 .. k0 + dk - 1 of ldk
    const int ldk = a.dk, k0 = PARTS ? kPartKeys * part : 0, dk = PARTS ? min(kPartKeys, ldk - k0) : ldk, dv = a.dv;
    const bool two = dk > 64;

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_TMEM);
    Ctl *ctl = reinterpret_cast<Ctl *>(sm + OFF_CTL);
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            mbar_init(&bar[i], i >= EMPTY_V && i < W_FREE ? WEIGHTS : 1);
        }
        *ctl = Ctl{sref.word, sref.stamp, timeout_ns, 0, 0, b};
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
    } else if (warp < WEIGHTS) {
        // 16-byte group (8 value rows) k8 of steps r32 and r32 + 32 of each half
        const int r32 = tid >> 3, k8 = tid & 7;
        const float *to_end = a.hd.to_end + ht::step_at(a, bh, s0) + r32;
        float wn[4] = {}, fn = 0.0f;   // the next chunk's, and what decays after it
        auto load = [&](int c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) wn[i] = __ldcg(to_end + c * C + 32 * i);
            fn = __ldcg(&reinterpret_cast<const ht::Chunk *>(ht::record_at(a, bh, s0 + int64_t(c) * C))->after);
        };
        if (n_chunks > 0) load(0);
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c % NS;
            unsigned char *V = sm + OFF_V + st * V_BYTES;
            const bool tail = c * C + C > nrun;
            float wc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) wc[i] = wn[i] * fn;
            if (c + 1 < n_chunks) load(c + 1);
            bool ok = hw(FULL_V + st, c / NS);
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
                    w[i] = hf == 0 ? wc[i] : wc[2 + i];
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
            if (lane == 0) arrive(&bar[EMPTY_V + st]);
        }
        // key column j, value rows 32 sh .. of the block's 64
        const int j = 32 * (warp & 3) + lane, sh = warp >> 2, i0 = vt * RB + 32 * sh;
        const bool done = n_chunks > 0 && __all_sync(0xffffffffu, hw(DONE, 0));
        tc_fence_after();
        const uint32_t D = tmem + 32 * sh + (uint32_t((warp & 3) * 32) << 16);
        const float f = dec::exp2_fix(a.seg_tot[size_t(bh) * nseg + seg]);
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
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
    const bool redo = ctl->redo != 0;
    if (tid == 0) a.seg_bad[(size_t(bh) * nseg + seg) * a.seg_tiles + (PARTS ? vt * a.parts + part : vt)] = redo;
    if (redo && ctl->abort_flag == 0) dt::redo_call<true, true>(a, ctl->row, n_vt, sm);
}

// ---------------------------------------------------------------------------
// PARTS: the block's part of the key columns, its outputs a term of the sum, which the sum
// gates; GATE: outputs are gated here; SKIP: there may be a skip (PARTS: in the first part's blocks)
template <bool PARTS, bool GATE, bool SKIP>
__global__ void __launch_bounds__(ht::THREADS, 1)
    heads_tensor_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_z,
                        const __grid_constant__ DecayArgs a, int n_vt, uint64_t timeout_ns, StatusRef sref) {
    using namespace ht;
    using bf = __nv_bfloat16;
    using Wt = Weights<GATE>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nseg = a.n_seg;
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
    const int b = dec::row_at(a, x / a.H, reinterpret_cast<int *>(sm + OFF_W)), bh = b * a.H + h;
    const int len = dec::row_len(a.lens, b, a.L);
    const int s0 = int(int64_t(seg) * a.seg_len);
    const int send = int(min(a.L, int64_t(s0) + a.seg_len));
    const int nrun = max(0, min(len, send) - s0);
    const int n_chunks = (nrun + C - 1) / C;
    // the block's key columns: k0 .. k0 + dk - 1 of ldk
    const int ldk = a.dk, k0 = PARTS ? kPartKeys * part : 0, dk = PARTS ? min(kPartKeys, ldk - k0) : ldk, dv = a.dv;
    const int nkk = (dk + 15) / 16;          // 16-wide steps over the key columns
    const bool two = dk > 64;                // two 64-column halves of Q and K
    const size_t g0 = step_at(a, bh, s0);    // the segment's gates
    const bool has_skip = SKIP && (!PARTS || (a.hd.skip != nullptr && part == 0));

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_TMEM);
    Ctl *ctl = reinterpret_cast<Ctl *>(sm + OFF_CTL);
    const Chunk *rec = reinterpret_cast<const Chunk *>(sm + OFF_G);
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            int n = 1;
            if (i >= F_DONE && i < K_DONE + 2) n = 8;
            if (i == DS_FREE || i == DS_FREE + 1 || i == EMPTY_Z || i == SB_READY || i == FIX) n = 8;
            // K is read by dS and P, Q by P and OX, V by the weight warps (through dS), by OI and,
            // with a skip, by the output warps
            if ((i >= EMPTY_Q && i < EMPTY_Q + 2) || (i >= EMPTY_K && i < EMPTY_K + 2) ||
                (i >= EMPTY_V && i < EMPTY_V + 2))
                n = 2;
            if (has_skip && i >= EMPTY_V && i < EMPTY_V + 2) n = 2 + 8;
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
    // What is read of the gates' launch waits for it; in a segmented call the launch
    // between has waited for it before this one could start, and segments past the
    // first wait for that one's states.
    auto gates_wait = [&]() {
        if (nseg == 1 || seg > 0) grid_dependency_wait();
    };

    if (warp == TMA_WARP) {   // --------------------------------------- TMA
        if (lane == 0) {
            prefetch_tensormap(&tm_q);
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
            if (GATE) prefetch_tensormap(&tm_z);
            auto load_qk = [&](int n, const CUtensorMap *tm, int off, int full) {
                const int st = n & 1, t = s0 + n * C;
                unsigned char *dst = sm + off + st * Q_BYTES;
                mbar_arrive_expect_tx(&bar[full + st], two ? 2 * HALF : HALF);
                tma_load_4d(dst, tm, &bar[full + st], k0, hk, t, b);
                if (two) tma_load_4d(dst + HALF, tm, &bar[full + st], k0 + 64, hk, t, b);
            };
            auto load_v = [&](int n) {
                const int st = n & 1;
                mbar_arrive_expect_tx(&bar[FULL_V + st], V_BYTES);
                tma_load_4d(sm + OFF_V + st * V_BYTES, &tm_v, &bar[FULL_V + st], vt * RB, h, s0 + n * C, b);
            };
            auto load_g = [&](int n) {
                const int st = n & 1;
                mbar_arrive_expect_tx(&bar[FULL_G + st], kChunkRecord);
                bulk_load(sm + OFF_G + st * kChunkRecord, record_at(a, bh, s0 + int64_t(n) * C), kChunkRecord,
                          &bar[FULL_G + st]);
            };
            auto load_z = [&](int n) {   // the one tile
                mbar_arrive_expect_tx(&bar[FULL_Z], V_BYTES);
                tma_load_4d(sm + OFF_Z, &tm_z, &bar[FULL_Z], vt * RB, h, s0 + n * C, b);
            };
            int nq = 0, nk = 0, nv = 0, ng = 0, nz = 0;
            for (; nv < 2 && nv < n_chunks; ++nv, ++nq, ++nk) {
                load_qk(nv, &tm_q, OFF_Q, FULL_Q);
                load_qk(nv, &tm_k, OFF_K, FULL_K);
                load_v(nv);
            }
            if (GATE && n_chunks > 0) load_z(nz), ++nz;
            gates_wait();
            fence_proxy_async_global();
            for (; ng < nv; ++ng) load_g(ng);
            // in the order in which a chunk lets go of them; once its last products (O's) have
            // let go of V nobody reads its record either
            for (int n = 2; n <= n_chunks; ++n) {
                const int st = n & 1, ph = (n - 2) >> 1;
                if (n < n_chunks) {
                    if (!hw(EMPTY_Q + st, ph)) break;
                    load_qk(n, &tm_q, OFF_Q, FULL_Q), ++nq;
                    if (!hw(EMPTY_K + st, ph)) break;
                    load_qk(n, &tm_k, OFF_K, FULL_K), ++nk;
                    if (!hw(EMPTY_V + st, ph)) break;
                    load_v(n), ++nv;
                    load_g(n), ++ng;
                }
                if (GATE) {
                    if (!hw(EMPTY_Z, n - 2)) break;
                    load_z(n - 1), ++nz;
                }
            }
            // copies still in flight land before the block exits
            auto land = [&](int full, int n) {
                for (int c = max(n - 2, 0); c < n; ++c) mbar_wait_bounded(&bar[full + (c & 1)], (c >> 1) & 1, timeout_ns);
            };
            land(FULL_Q, nq);
            land(FULL_K, nk);
            land(FULL_V, nv);
            land(FULL_G, ng);
            if (nz > 0) mbar_wait_bounded(&bar[FULL_Z], (nz - 1) & 1, timeout_ns);
        }
    } else if (warp >= DS_WARP) {   // -------------------------------- products
        // every wait's answer is made warp-uniform, and so is all that follows
        auto hu = [&](int i, int phase) -> bool { return __all_sync(0xffffffffu, hw(i, phase)); };
        const bool lead = elect_one();
        const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
        if (warp == DS_WARP) {
            const uint64_t dW = umma_smem_desc(base + OFF_W, HALF, 1024);
            for (int c = 0; c < n_chunks; ++c) {
                const int st = c & 1;
                // the last dS in these columns has been read
                if (!hu(FULL_K + st, c >> 1) || (c >= 2 && !hu(DS_FREE + st, (c - 2) >> 1))) break;
                const uint64_t dK = umma_smem_desc(base + OFF_K + st * Q_BYTES, HALF, 1024);
                bool ok = true;
#pragma unroll 1
                for (int e = 0; e < 4 * Wt::HALVES; ++e) {   // quarters, or their first halves, then their second ones
                    const int qt = e & 3, hf = e >> 2;
                    ok = ok && hu(W_READY + qt, Wt::HALVES * c + hf);
                    if (!ok) break;
                    tc_fence_after();
                    if (lead) {   // 16 steps are 2048 bytes on, 128 in the descriptors' units
                        // the three terms onto one accumulator, small ones first
#pragma unroll
                        for (int kk = 0; kk < Wt::STEPS / 16; ++kk)
#pragma unroll
                            for (int term = 2; term >= 0; --term)
                                umma_bf16(tmem + T_DS + st * 64, dK + 256 * qt + 128 * (hf + kk),
                                          dW + (Wt::TERM >> 4) * term + 8 * Wt::STEPS * qt + 128 * kk, IDESC_DS,
                                          e > 0 || kk > 0 || term < 2);
                        umma_commit(&bar[W_FREE + qt]);
                        if (e == 4 * Wt::HALVES - 1) {
                            umma_commit(&bar[DS_DONE + st]);
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
        } else {
            const uint64_t dS = umma_smem_desc(base + OFF_SB, HALF, 1024);
            int n_steep = 0;
            for (int c = 0; c < n_chunks; ++c) {
                const int st = c & 1;
                // the state before chunk c; chunk c - 2's outputs have been read
                if (!hu(SB_READY, c) || !hu(FULL_Q + st, c >> 1)) break;
                if (c >= 2 && !hu(K_DONE + st, (c - 2) >> 1)) break;
                tc_fence_after();
                const uint64_t dQ = umma_smem_desc(base + OFF_Q + st * Q_BYTES, 16, 1024);
                if (lead) {
#pragma unroll 1
                    for (int kk = 0; kk < nkk; ++kk)
                        umma_bf16(tmem + T_O + st * 64, dQ + (((kk >> 2) * HALF + (kk & 3) * 32) >> 4), dS + 128 * kk, IDESC_O,
                                  kk > 0);
                    umma_commit(&bar[OX_DONE + st]);
                    umma_commit(&bar[EMPTY_Q + st]);
                }
                __syncwarp();
                if (!hu(F_DONE + st, c >> 1) || !hu(FULL_V + st, c >> 1)) break;
                if (!hu(FULL_G + st, c >> 1) || (rec[st].steep != 0 && !hu(FIX, n_steep++))) break;
                // the last chunk: V's rows past the end have been zeroed for dS
                if (c * C + C > nrun && !hu(DS_DONE + st, c >> 1)) break;
                tc_fence_after();
                const uint64_t dV = umma_smem_desc(base + OFF_V + st * V_BYTES, HALF, 1024);
                if (lead) {   // onto Q S^T: same shape and accumulator, so in order
#pragma unroll 1
                    for (int kk = 0; kk < C / 16; ++kk)
                        umma_bf16_ts(tmem + T_O + st * 64, tmem + T_P + st * 128 + 16 * kk, dV + 128 * kk,
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
    } else if (is_weight(warp)) {   // ---------------------------------- weight
        // lane: a step of the quarter; or, i and i + 16, step i of half of it, 32 value columns each
        const int qt = warp == 20 ? 0 : warp - 23, i = lane % Wt::STEPS, wh = lane / Wt::STEPS, r = Wt::STEPS * qt + i;
        gates_wait();
        const float *src = a.hd.weight + g0 + 32 * qt + i;
        float wn = n_chunks > 0 ? __ldcg(src) : 0.0f;
        for (int p = 0; p < Wt::HALVES * n_chunks; ++p) {
            const int c = p / Wt::HALVES, hf = p % Wt::HALVES, st = c & 1, s = 32 * qt + 16 * hf + i;   // s: of the chunk
            unsigned char *V = sm + OFF_V + st * V_BYTES;
            const bool in = c * C + s < nrun;
            const float w = wn;
            if (p + 1 < Wt::HALVES * n_chunks) wn = __ldcg(src + (p + 1) / Wt::HALVES * C + 16 * ((p + 1) % Wt::HALVES));
            bool ok = hw(FULL_V + st, c >> 1);
            if (ok && c * C + C > nrun) ok = hw(FULL_K + st, c >> 1);
            if (ok && p >= 1) ok = hw(W_FREE + qt, p - 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t from = sw128_offset(s, 32 * wh), to = OFF_W + sw128_offset(r, 32 * wh);
#pragma unroll 1
            for (int k = 0; k < Wt::GROUPS; ++k) {   // 8 columns
                uint4 u = *reinterpret_cast<const uint4 *>(V + (from ^ (k << 4)));
                if (!in) u = make_uint4(0, 0, 0, 0);
                const uint32_t uv[4] = {u.x, u.y, u.z, u.w};
                uint32_t t1[4], t2[4], t3[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) three_terms(w, uv[e], t1[e], t2[e], t3[e]);
                unsigned char *W = sm + (to ^ (k << 4));
                *reinterpret_cast<uint4 *>(W) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                *reinterpret_cast<uint4 *>(W + Wt::TERM) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                *reinterpret_cast<uint4 *>(W + 2 * Wt::TERM) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
            }
            if (!in) {   // past the row's end: whatever stands there must not reach a product
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int k = 0; k < Wt::GROUPS; ++k) {
                    const uint32_t at = s * 128 + 64 * wh + 16 * k;
                    *reinterpret_cast<uint4 *>(V + at) = z;
                    *reinterpret_cast<uint4 *>(sm + OFF_K + st * Q_BYTES + at) = z;
                    if (two) *reinterpret_cast<uint4 *>(sm + OFF_K + st * Q_BYTES + HALF + at) = z;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&bar[W_READY + qt]);
        }
    } else if (warp >= FRONT) {   // ------------------------------------- front
        // Rows 32 fw .. of P, blocks of 16 columns first .. end of those that some row sees; the
        // others are cleared.  A block's PD goes to the first half of its own columns.
        const int fw = warp & 3, k = warp == 27 ? 2 : (warp - FRONT) >> 2, t = 32 * fw + lane;
        const int seen = 2 * fw + 2, sharers = fw == 0 ? 1 : fw == 3 ? 3 : 2, each = (seen + sharers - 1) / sharers;
        const int first = k * each, end = min(seen, first + each);
        const int clear = (8 - seen) / sharers, clear0 = seen + k * clear;   // (evenly shared)
        gates_wait();
        const float2 *src = a.hd.own + g0 + t;
        float2 next = n_chunks > 0 ? __ldcg(src) : make_float2(0.0f, 0.0f);
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c & 1;
            const uint32_t P = tmem + T_P + st * 128 + (uint32_t(fw * 32) << 16);
            const float2 own = next;
            if (c + 1 < n_chunks) next = __ldcg(src + (c + 1) * C);
            const bool ok = hw(FULL_G + st, c >> 1) && hw(P_READY + st, c >> 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const bool cut = nrun - c * C < C;
            const bool steep = rec[st].steep != 0;
            const float *f = rec[st].col;
            const int lt = __float_as_int(own.y);               // steep
#pragma unroll 1
            for (int kb = clear0; kb < clear0 + clear; ++kb) {
                const uint32_t r[8] = {};
                tmem_st8_nowait(P + 16 * kb, r);
            }
#pragma unroll 1
            for (int kb = first; kb < end; ++kb) {
                const int b0 = 16 * kb;   // the block's first column
                uint32_t r[8];
                const bool diag = b0 + 15 > 32 * fw;   // it holds some row's diagonal
                float p[16];
                tmem_ld16_nowait(P + 16 * kb, p);
                if (steep && diag) {
                    tmem_ld_wait_tied(p);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {   // the warp's own steps
                        const int from = (b0 & 16) + e;
                        const float ds = __shfl_sync(0xffffffffu, own.x, from);
                        const int ls = __shfl_sync(0xffffffffu, lt, from);
                        // (a step past the row's is cut below; its power may be any)
                        p[e] = p[e] * ds * ex2_approx(dec::units_f(min(lt - ls, 0)));
                    }
                } else {
                    // rows past a steep chunk's block: as one factor more
                    const float rf = steep ? ex2_approx(dec::units_f(lt - rec[st].last[b0 >> 4])) : 1.0f;
                    float4 w4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w4[e] = *reinterpret_cast<const float4 *>(f + b0 + 4 * e);
                    tmem_ld_wait_tied(p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y0 = __fmul2_rn(make_float2(p[4 * e], p[4 * e + 1]), make_float2(w4[e].x, w4[e].y));
                        const float2 y1 =
                            __fmul2_rn(make_float2(p[4 * e + 2], p[4 * e + 3]), make_float2(w4[e].z, w4[e].w));
                        p[4 * e] = y0.x, p[4 * e + 1] = y0.y, p[4 * e + 2] = y1.x, p[4 * e + 3] = y1.y;
                    }
                    if (steep) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 y = __fmul2_rn(make_float2(p[e], p[e + 1]), make_float2(rf, rf));
                            p[e] = y.x, p[e + 1] = y.y;
                        }
                    }
                }
                if (diag) {   // row t sees columns up to its own
                    const int d = t - b0;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (e > d) p[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = pack(p[2 * e], p[2 * e + 1]);
                if (cut) {   // no columns past the row's end, whatever they hold
                    const int m = nrun - c * C - b0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[e] &= 2 * e + 1 < m ? 0xffffffffu : 2 * e < m ? 0xffffu : 0u;
                }
                tmem_st8_nowait(P + b0, r);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&bar[F_DONE + st]);
        }
    } else if (warp >= OUT) {   // --------------------------------------- output
        // row 32 (warp & 3) + lane of the chunk, value columns 32 oh ..
        const int row = 32 * (warp & 3) + lane, oh = (warp - OUT) >> 2, odd = lane & 1;
        const int i0 = vt * RB + 32 * oh;
        const size_t HV = size_t(a.H) * dv;
        bf *ob = static_cast<bf *>(a.o) + (size_t(b) * a.L + s0) * HV + size_t(h) * dv + i0;
        const float skip = has_skip ? a.hd.skip[h] : 0.0f;
        gates_wait();
        const float *src = a.hd.readout + g0 + row;
        float next = n_chunks > 0 ? __ldcg(src) : 0.0f;
        float2 zero = make_float2(0.0f, 0.0f);
        const uint32_t at = sw128_offset(row, 32 * oh);   // this thread's part of the tiles of V and of the gate
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c & 1;
            const uint32_t O = tmem + T_O + st * 64 + 32 * oh + (uint32_t((warp & 3) * 32) << 16);
            float u = next;
            if (c + 1 < n_chunks) next = __ldcg(src + (c + 1) * C);
            const int t = c * C + row;
            const bool valid = t < nrun;
            uint4 x[4] = {};   // 8 columns each
            if (SKIP && has_skip) {
                if (!__all_sync(0xffffffffu, hw(FULL_V + st, c >> 1))) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = read_now(sm + OFF_V + st * V_BYTES + (at ^ (16 * k)));
                __syncwarp();
                if (lane == 0) arrive(&bar[EMPTY_V + st]);
            }
            if (__float_as_int(u) < 0) {   // steep: rows of Q S^T by 2^(base + L) before PD V is added
                if (!__all_sync(0xffffffffu, hw(OX_DONE + st, c >> 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < 32; q += 16) {
                    float d[16];
                    tmem_ld16_nowait(O + q, d);
                    tmem_ld_wait_tied(d);
                    uint32_t w[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) w[r] = __float_as_uint(-u * d[r]);
                    tmem_st16_nowait(O + q, w);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&bar[FIX]);
                u = 1.0f;
            }
            bool there = hw(O_DONE + st, c >> 1);
            if (GATE && there) there = hw(FULL_Z, c);
            if (!__all_sync(0xffffffffu, there)) break;
            tc_fence_after();
            const float2 u2 = make_float2(u, u), s2 = make_float2(skip, skip);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float d[16];
                tmem_ld16_nowait(O + 16 * q, d);
                tmem_ld_wait_tied(d);
                if (q == 1) {   // the accumulator is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(&bar[K_DONE + st]);
                }
                const uint32_t xw[8] = {x[2 * q].x,     x[2 * q].y,     x[2 * q].z,     x[2 * q].w,
                                        x[2 * q + 1].x, x[2 * q + 1].y, x[2 * q + 1].z, x[2 * q + 1].w};
                auto out = [&](int r) {   // values 2 r and 2 r + 1 before the gate
                    float2 y = __fmul2_rn(u2, make_float2(d[2 * r], d[2 * r + 1]));
                    if (SKIP) y = __ffma2_rn(s2, make_float2(lo_f(xw[r]), hi_f(xw[r])), y);
                    return y;
                };
                const int col = i0 + 16 * q;
                if (PARTS) {   // steps past the row's end are the sum's to clear
                    float *dst = a.o_part + ((size_t(part) * a.B + b) * a.L + s0 + t) * HV + size_t(h) * dv + col;
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const float2 y0 = out(r / 2), y1 = out(r / 2 + 1);
                        const float4 y = make_float4(y0.x, y0.y, y1.x, y1.y);
                        if (valid && col + r < dv) *reinterpret_cast<float4 *>(dst + r) = y;
                        if (valid) zero.x = fmaf(0.0f, y.x, fmaf(0.0f, y.y, fmaf(0.0f, y.z, fmaf(0.0f, y.w, zero.x))));
                    }
                    continue;
                }
                uint32_t w[8];
                if constexpr (GATE) {
                    const uint4 lo = read_now(sm + OFF_Z + (at ^ (32 * q)));
                    const uint4 hi = read_now(sm + OFF_Z + (at ^ (32 * q + 16)));
                    if (q == 1) {   // the tile is free
                        __syncwarp();
                        if (lane == 0) arrive(&bar[EMPTY_Z]);
                    }
                    const uint32_t zw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        float2 y = out(r);
                        if (valid) zero = __ffma2_rn(y, make_float2(0.0f, 0.0f), zero);
                        y = __fmul2_rn(y, silu2_f(make_float2(lo_f(zw[r]), hi_f(zw[r]))));
                        w[r] = pack(y.x, y.y);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float2 y = out(r);
                        if (valid) zero = __ffma2_rn(y, make_float2(0.0f, 0.0f), zero);
                        w[r] = pack(y.x, y.y);
                    }
                }
                // whole 32-byte sectors: each lane stores 16 bytes of both rows of the pair
                uint4 lo = make_uint4(w[0], w[1], w[2], w[3]), hi = make_uint4(w[4], w[5], w[6], w[7]);
                if (!valid) lo = hi = make_uint4(0, 0, 0, 0);
                const uint4 mine = odd ? hi : lo, got = xor1(odd ? lo : hi);
                bf *dst = ob + size_t(t - odd) * HV + 16 * q + 8 * odd;   // the pair's first row
                if (col + 8 * odd < dv) {
                    if (s0 + t - odd < send) *reinterpret_cast<uint4 *>(dst) = odd ? got : mine;
                    if (s0 + t - odd + 1 < send) *reinterpret_cast<uint4 *>(dst + HV) = odd ? mine : got;
                }
            }
        }
        if (not_finite(zero)) ctl->redo = 1;
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
        gates_wait();
        if (seg > 0) {
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
            const int st = c & 1;
            bool ok = hw(FULL_G + st, c >> 1);
            // the bf16 copy's buffer is free
            if (ok && c >= 1) ok = hw(OX_DONE + ((c - 1) & 1), (c - 1) >> 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            const float m = rec[st].m;
            // a rescale belongs before the copy (the chunk's weights assume it) but
            // after it in a steep chunk, which applies its factors by rows
            const bool steep = rec[st].steep != 0;
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
            if (!__all_sync(0xffffffffu, hw(DS_DONE + st, c >> 1))) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 32; q += 16) {
                float d[16];
                tmem_ld16_nowait(D + st * 64 + q, d);
                tmem_ld_wait_tied(d);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 z = __fadd2_rn(make_float2(S[q + e], S[q + e + 1]), make_float2(d[e], d[e + 1]));
                    S[q + e] = z.x, S[q + e + 1] = z.y;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&bar[DS_FREE + st]);
        }
        float *out = seg == a.n_seg - 1 && a.S_final != nullptr ? a.S_final + size_t(bh) * dv * ldk + k0 : nullptr;
        if (out != nullptr && j < dk) {
            const float f = __ldcg(a.hd.left + size_t(bh) * nseg + seg);
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
            dt::redo_block<false, true>(a, ctl->row, n_vt, sm);
        else
            dt::redo_call<false, true>(a, ctl->row, n_vt, sm);
    }
}

namespace {

bool ht_setup() {
    static DeviceSetup setup;
    return setup.run([] {
        auto room = [](auto kern, uint32_t bytes) {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == cudaSuccess;
        };
        return room(heads_state_kernel<false>, hs::SMEM) && room(heads_state_kernel<true>, hs::SMEM) &&
               room(heads_tensor_kernel<false, false, false>, ht::SMEM) &&
               room(heads_tensor_kernel<false, false, true>, ht::SMEM) &&
               room(heads_tensor_kernel<false, true, false>, ht::SMEM) &&
               room(heads_tensor_kernel<false, true, true>, ht::SMEM) &&
               room(heads_tensor_kernel<true, false, true>, ht::SMEM);
    });
}

}  // namespace

int heads_tensor_launch(const DecayArgs &a, StatusRef st, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mz;
    if (!dt_map(&mq, a.q, a.dk, a.Hk, a.L, a.B, a.hd.ldq) || !dt_map(&mk, a.k, a.dk, a.Hk, a.L, a.B, a.hd.ldk) ||
        !dt_map(&mv, a.v, a.dv, a.H, a.L, a.B, a.hd.ldv) || !ht_setup())
        return LR_ERR_CUDA;
    mz = mv;   // (not read without a gate)
    if (a.hd.z != nullptr && !dt_map(&mz, a.hd.z, a.dv, a.H, a.L, a.B, a.hd.ldz)) return LR_ERR_CUDA;
    const int n_vt = (a.dv + ht::RB - 1) / ht::RB;
    const bool parts = a.parts > 1;
    const int64_t per_seg = a.B * a.H * n_vt * a.parts;
    if (per_seg * a.n_seg > INT32_MAX) return LR_ERR_UNSUPPORTED;
    const int64_t chunks = (a.seg_len + ht::C - 1) / ht::C;
    int rc = launch_early(heads_gates_kernel, dim3(unsigned(a.B * a.H * a.n_seg)), int(32 * (chunks < 32 ? chunks : 32)),
                          stream, a, st);
    if (rc == LR_OK && a.n_seg > 1)
        rc = launch_kernel(parts ? heads_state_kernel<true> : heads_state_kernel<false>, true,
                           dim3(unsigned(per_seg * (a.n_seg - 1))), hs::THREADS, hs::SMEM, stream, mk, mv, a, n_vt,
                           dt::wait_limit_ns(), st);
    const bool z = a.hd.z != nullptr, skip = a.hd.skip != nullptr;
    if (rc == LR_OK)
        rc = launch_kernel(parts ? heads_tensor_kernel<true, false, true>
                           : z   ? (skip ? heads_tensor_kernel<false, true, true> : heads_tensor_kernel<false, true, false>)
                                 : (skip ? heads_tensor_kernel<false, false, true> : heads_tensor_kernel<false, false, false>),
                           true,
                           dim3(unsigned(per_seg * a.n_seg)), ht::THREADS, ht::SMEM, stream, mq, mk, mv, mz, a, n_vt,
                           dt::wait_limit_ns(), st);
    if (rc != LR_OK || !parts) return rc;
    const int64_t rows = a.B * a.L;
    return launch_early(decay_parts_kernel<true>, dim3(unsigned(rows < (1 << 20) ? rows : 1 << 20)), 256, stream, a);
}

}  // namespace lr
