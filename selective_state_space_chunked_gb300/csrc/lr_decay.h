// lr_decay.h -- host-side declarations of the decayed linear attention
// (lr_decay_attn_fwd): the call's arguments, its plan and the two launchers.
#pragma once

#include "lr_internal.h"

namespace lr {

// What a selective scan with heads has beside the decayed attention (HEADS kernels,
// with q = C, k = B, v = x, g = dt, a_log = A_log, o = y; see lr_selective_heads_fwd):
//   delta_t = softplus(dt_t + dt_bias),  log decay -exp(A_log) delta_t,
//   S_t = a_t S_{t-1} + delta_t x_t B_t^T,  y_t = (S_t C_t + skip x_t) silu(z_t)
// and inputs whose rows lie ld* elements apart.
struct HeadsArgs {
    const float *dt_bias;    // (H) or NULL
    const float *skip;       // (H) or NULL
    const void *z;           // like v, or NULL
    int64_t ldq, ldk, ldv, ldg, ldz;
    int softplus;
    // Tensor cores: what a first launch makes of the gates (lr_heads_tensor.cu), for
    // every step of every (batch row, head), in whole chunks, and for every chunk.
    float *weight, *readout, *to_end;
    float2 *own;
    unsigned char *chunk;
    float *left;             // [batch row, head][segment]
};
constexpr int kChunkRecord = 576;   // bytes of a chunk's


// One call, as its kernels see it (device pointers; see lr_decay_attn_fwd).
struct DecayArgs {
    const void *q, *k, *v;
    const float *a_log;      // (H) or NULL
    const void *g;           // (B, L, H) io or NULL
    const int32_t *lens;     // (B) or NULL
    const float *S0;         // (B, H, dv, dk) or NULL
    void *o;
    float *S_final;          // or NULL
    int64_t B, L;
    int H, Hk, dk, dv;
    float scale;
    // Time segments: every (batch row, head) is cut into n_seg ranges of
    // seg_len steps.  With more than one, a first launch leaves the state
    // that each range but the last builds from its own steps (range 0 from
    // S0) in seg_state [(b H + h)(n_seg - 1) + s][dv][dk] and its log2 decay,
    // in units of 2^-32, in seg_tot; the second launch starts every range
    // from the decayed sum of the ranges before it.  seg_bad
    // [((b H + h)(n_seg - 1) + s) seg_tiles + tile]: whether a block's tile of such a state
    // holds an infinity or a NaN, which no decay ends.
    int n_seg, seg_tiles;
    int64_t seg_len;
    float *seg_state;
    long long *seg_tot;
    int *seg_bad;
    // Tensor cores, dk > 128: the key columns in parts of kPartKeys, each a
    // recurrence of its own with the same decays; their outputs, fp32, in
    // o_part [part][B][L][H][dv], are summed by a last launch.
    int parts;
    float *o_part;
    bool by_length;          // blocks take the batch rows by falling length
    HeadsArgs hd;            // HEADS kernels alone
};

struct DecayPlan {
    int path = 0;            // 0: CUDA cores, 1: tensor cores
    int n_seg = 1;
    int64_t seg_len = 0;
    int thread_rows = 4;     // CUDA cores: state rows per thread
    int parts = 1;
    int tiles = 1;           // blocks of one (batch row, head, segment)
    int64_t blocks = 0;      // of the (second) launch
    size_t ws_bytes = 0;     // status, then seg_tot, seg_bad, seg_state, o_part
};

// heads: a selective scan with heads (a.hd)
int decay_plan(int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv, lr_dtype io, bool heads,
               DecayPlan *p);
int decay_attn_launch(DecayArgs a, lr_dtype io, const DecayPlan &p, bool heads, void *workspace, cudaStream_t stream);

// CUDA-core kernel, one translation unit per I/O type
template <typename IO, bool HEADS>
int decay_general_launch(const DecayArgs &a, const DecayPlan &p, StatusRef st, cudaStream_t stream);
// tensor-core kernels: bf16 I/O, dk and dv multiples of 8
int decay_tensor_launch(const DecayArgs &a, StatusRef st, cudaStream_t stream);
int heads_tensor_launch(const DecayArgs &a, StatusRef st, cudaStream_t stream);
constexpr int kOrderRows = 64;      // the largest batch that is taken by length
constexpr int kDecayChunk = 128;    // its steps per chunk (segments are multiples of it)
constexpr int kDecayRows = 64;      // its value rows per block
constexpr int kPartKeys = 128;      // its key columns per block
// rows of the state per block of the general kernel
int decay_general_rows(int64_t dk, int thread_rows);

// One launch, and its own status: an error that an earlier call of the thread left
// unread says nothing about it (a caller that is told of a failure may launch
// again, onto a state that has been updated).  early: it may start while the kernel
// before it on the stream drains, and waits for that one's results itself
// (grid_dependency_wait).
template <typename... P, typename... A>
int launch_kernel(void (*kern)(P...), bool early, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, P(args)...) == cudaSuccess) return LR_OK;
    (void)cudaGetLastError();   // reported here
    return LR_ERR_CUDA;
}
template <typename... P, typename... A>
int launch_early(void (*kern)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
    return launch_kernel(kern, true, grid, threads, 0, stream, args...);
}

// hd: a selective scan with heads, or NULL
int decay_step_launch(const void *q, const void *k, const void *v, const float *a_log, const void *g,
                      float scale, const float *S_in, float *S_out, void *o, int64_t B, int64_t H, int64_t Hk,
                      int64_t dk, int64_t dv, int io_bf16, const HeadsArgs *hd, cudaStream_t stream);

int group_norm_act_launch(const void *x, const void *z, const float *gamma, const float *beta, void *y,
                          int64_t N, int64_t C, int64_t G, float eps, int act, int io_bf16, cudaStream_t stream);

int causal_conv_launch(const void *x, int64_t ldx, const float *w, const float *bias, const void *state,
                       const int32_t *lens, void *y, void *state_out, int64_t B, int64_t L, int64_t C, int W, int act,
                       int io_bf16, bool step, cudaStream_t stream);

int head_norm_rope_launch(const void *q, int64_t ldq, const void *k, int64_t ldk, const float *gq, const float *gk,
                          const float *freqs, const int32_t *pos, void *qo, void *ko, int64_t N, int64_t H, int64_t Hk,
                          int64_t d, int64_t rot, int norm, float eps, int pairs, int io_bf16, cudaStream_t stream);

}  // namespace lr
