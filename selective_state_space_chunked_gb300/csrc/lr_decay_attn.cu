// lr_decay_attn.cu -- plan and dispatch of the decayed linear attention.
#include "lr_decay.cuh"

namespace lr {

namespace {
// CUDA-core kernel: blocks that fill the GPU (four of 128 threads per SM: their
// state registers), and the shortest segment worth the second pass over k and v.
constexpr int64_t kGenBlocksPerSm = 4;
constexpr int64_t kGenMinSeg = 128;
constexpr int64_t kMaxSeg = 32;
// Tensor-core kernel: the shortest sequence it takes, and costs in units of a
// chunk's time: a chunk of the first launch, a block's start, and one
// segment's state read by a later one.
constexpr int64_t kTensorMinLen = 64;
constexpr double kFirstCost = 0.6, kBlockCost = 3.0, kStateCost = 0.5;
}  // namespace

int decay_plan(int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv, lr_dtype io, DecayPlan *p) {
    (void)Hk;
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    int64_t n = 1, unit = 16;
    p->narrow = false;
    p->path = io == LR_BF16 && dk <= 128 && dk % 8 == 0 && dv % 8 == 0 && L >= kTensorMinLen;
    if (p->path == 1) {
        // one block per SM: waves of blocks, each as long as its chunks and a
        // block's start
        unit = kDecayChunk;
        const int64_t chunks = (L + unit - 1) / unit, blocks = B * H * ((dv + kDecayRows - 1) / kDecayRows);
        auto waves = [&](int64_t b) { return double((b + sms - 1) / sms); };
        double best = waves(blocks) * (double(chunks) + kBlockCost);
        for (int64_t s = 2; s <= kMaxSeg && 2 * s <= chunks; ++s) {
            const double per = double((chunks + s - 1) / s);
            const double t = waves(blocks * s) * (per + kBlockCost + kStateCost * double(s)) +
                             waves(blocks * (s - 1)) * (kFirstCost * per + kBlockCost);
            if (t < best) best = t, n = s;
        }
    } else {
        const int64_t want = kGenBlocksPerSm * sms;
        auto blocks = [&](bool narrow) {
            const int64_t rows = decay_general_rows(dk, narrow);
            return B * H * ((dv + rows - 1) / rows);
        };
        n = want / blocks(false);
        if (n > L / kGenMinSeg) n = L / kGenMinSeg;
        if (n > kMaxSeg) n = kMaxSeg;
        if (n < 1) n = 1;
        p->narrow = n == 1 && blocks(false) < sms;
    }
    p->seg_len = ((L + n - 1) / n + unit - 1) / unit * unit;
    p->n_seg = int((L + p->seg_len - 1) / p->seg_len);
    const size_t segs = size_t(B) * H * (p->n_seg - 1);
    p->ws_bytes = kStatusBytes + (segs * sizeof(long long) + 15) / 16 * 16 + segs * dv * dk * sizeof(float);
    return LR_OK;
}

int decay_attn_launch(DecayArgs a, lr_dtype io, const DecayPlan &p, void *workspace, cudaStream_t stream) {
    unsigned char *ws = static_cast<unsigned char *>(workspace) + kStatusBytes;
    const size_t segs = size_t(a.B) * a.H * (p.n_seg - 1);
    a.n_seg = p.n_seg;
    a.seg_len = p.seg_len;
    a.seg_tot = reinterpret_cast<long long *>(ws);
    a.seg_state = reinterpret_cast<float *>(ws + (segs * sizeof(long long) + 15) / 16 * 16);
    const StatusRef st = call_status(workspace);
    if (p.path == 1) return decay_tensor_launch(a, st, stream);
    return io == LR_BF16 ? decay_general_launch<__nv_bfloat16>(a, p, st, stream)
                         : decay_general_launch<float>(a, p, st, stream);
}

}  // namespace lr
