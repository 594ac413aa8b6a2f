// lr_decay_attn.cu -- plan and dispatch of the decayed linear attention.
#include "lr_decay.cuh"

namespace lr {

namespace {
// CUDA-core kernel: the shortest segment, and costs in units of a step of a
// block: a block's start, one segment's state read by a later one, and the
// second launch.  Chosen on sweeps of the segment count over 20 shapes.  fp32
// H16 d128 (of a kernel 5 % slower), B2 L2048: 4 segments 271 us, 7 242, 9 (chosen)
// 210, 12 246; B4 L4096: 1 999, 4 748, 9 (chosen) 682, 14 690; B1 L32768: 9 1821,
// 19 (chosen) 1304, 24 1490; few heads: B1 L8192 H1 d128 32 114, 64 (chosen) 72, 96
// 88; B1 L4096 H2 d64 32 57, 45 (chosen) 47, 64 68.
// Calls in one segment whose narrow blocks (one state row a thread) are no more
// than four per SM, with fp32 I/O and more than 64 keys three, take those.  L100 fp32:
// d128 H4 20.2 us against 28.2, H16 21.0 against 28.5, H28 23.5 against 28.2, H32 32.8
// against 28.2; d64 H16 15.0 against 20.1, H76 19.5 against 20.2; dk 256 H12 24.7
// against 27.4, H16 44.0 against 27.5.  bf16 L32 d128: H4 8.0 against 11.0, H32 8.5
// against 10.6.  (At dk 256, bf16 L32 24.2 against 12.1, and at dk 512, fp32 98
// against 41, when the narrow form came in.)
constexpr int64_t kGenMinSeg = 64;
constexpr double kGenBlockCost = 40.0, kGenStateCost = 3.0, kGenLaunchCost = 50.0;
constexpr int64_t kGenMaxSeg = 96;
// Tensor-core kernel: the shortest sequence it takes (bf16, on it and on the CUDA
// cores: B1 L48 H4 d128 10.7 and 11.7 us, L32 10.5 and 8.2; B4 L48 H32 d64 11.0 and
// 14.4; B1 H8 dk256, L48 13.1 and 16.2, L32 13.2 and 12.1; the other way, B8 L48 H16
// d128 21.9 and 19.1), and costs in units of a chunk's time: a chunk of the first
// launch, a block's start, and one segment's state read by a later one.  Against
// sweeps of the segment count over 11 shapes the plan's choice is the best or
// within 3 %: B1 L32768 H16 d128 1 segment 582 us, 2 447, 4 (chosen) 238, 8 256;
// B1 L16384 H8 dk64 6 84, 8 69, 9 (chosen) 66, 12 95; B4 L2048 H16 1 (chosen) 49.5,
// 2 74.
constexpr int64_t kMaxSeg = 32;
constexpr int64_t kTensorMinLen = 48;
constexpr double kFirstCost = 0.6, kBlockCost = 3.0, kStateCost = 1.0;
}  // namespace

namespace {
size_t tot_bytes(size_t segs) { return (segs * sizeof(long long) + 15) / 16 * 16; }
size_t bad_bytes(size_t segs, const DecayPlan &p) { return (segs * p.tiles * sizeof(int) + 15) / 16 * 16; }
}  // namespace

int decay_plan(int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv, lr_dtype io, DecayPlan *p) {
    (void)Hk;
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    int64_t n = 1, unit = 16;
    p->narrow = false;
    p->path = io == LR_BF16 && dk % 8 == 0 && dv % 8 == 0 && L >= kTensorMinLen;
    p->parts = p->path == 1 ? int((dk + kPartKeys - 1) / kPartKeys) : 1;
    if (p->path == 1) {
        // one block per SM: waves of blocks, each as long as its chunks and a
        // block's start
        unit = kDecayChunk;
        const int64_t chunks = (L + unit - 1) / unit, blocks = B * H * ((dv + kDecayRows - 1) / kDecayRows) * p->parts;
        auto waves = [&](int64_t b) { return double((b + sms - 1) / sms); };
        double best = waves(blocks) * (double(chunks) + kBlockCost);
        for (int64_t s = 2; s <= kMaxSeg && 2 * s <= chunks; ++s) {
            const double per = double((chunks + s - 1) / s);
            const double t = waves(blocks * s) * (per + kBlockCost + kStateCost * double(s)) +
                             waves(blocks * (s - 1)) * (kFirstCost * per + kBlockCost);
            if (t < best) best = t, n = s;
        }
    } else {
        // Blocks of an SM share its fp32 pipes.  The SM with the most of them
        // takes, per step and in units of a block's share of a full SM, as long
        // as its slots for each full round (a partly filled last round of
        // dependent launches packs three blocks as four), 2 where no SM has a
        // second block (a step then takes 0.243 us against 0.49 for four blocks),
        // and 1.5 for a block left over by the rounds, whose start overlaps them.
        const int64_t rows = decay_general_rows(dk, false), threads = dk <= 64 ? 64 : 128, slots = dk <= 128 ? 4 : 3;
        const int64_t blocks = B * H * ((dv + rows - 1) / rows);
        auto load = [&](int64_t b) {
            const int64_t most = (b * threads + 128 * sms - 1) / (128 * sms), rest = most % slots;
            if (most == 1) return 2.0;
            return double(most - rest) + (rest == 0 ? 0.0 : rest == 1 ? 1.5 : rest == 2 ? 2.75 : double(slots));
        };
        double best = load(blocks) * (double(L) + kGenBlockCost);
        for (int64_t s = 2; s <= kGenMaxSeg && s * kGenMinSeg <= L; ++s) {
            const double per = double((L + s - 1) / s);
            const double t = load(blocks * s) * (per + kGenBlockCost + kGenStateCost * double(s)) +
                             load(blocks * (s - 1)) * (0.5 * per + kGenBlockCost) + kGenLaunchCost;
            if (t < best) best = t, n = s;
        }
        const int64_t nrows = decay_general_rows(dk, true);
        const int64_t narrow_per_sm = io == LR_BF16 || dk <= 64 ? 4 : 3;
        p->narrow = n == 1 && dk <= (io == LR_BF16 ? 128 : 256) && B * H * ((dv + nrows - 1) / nrows) <= narrow_per_sm * sms;
    }
    p->seg_len = ((L + n - 1) / n + unit - 1) / unit * unit;
    p->n_seg = int((L + p->seg_len - 1) / p->seg_len);
    const int64_t rows = p->path == 1 ? kDecayRows : decay_general_rows(dk, p->narrow);
    p->tiles = int((dv + rows - 1) / rows) * p->parts;
    p->blocks = B * H * p->tiles * p->n_seg;
    const size_t segs = size_t(B) * H * (p->n_seg - 1);
    p->ws_bytes = kStatusBytes + tot_bytes(segs) + bad_bytes(segs, *p) + segs * dv * dk * sizeof(float);
    if (p->parts > 1) p->ws_bytes += size_t(p->parts) * B * L * H * dv * sizeof(float);
    return LR_OK;
}

int decay_attn_launch(DecayArgs a, lr_dtype io, const DecayPlan &p, void *workspace, cudaStream_t stream) {
    unsigned char *ws = static_cast<unsigned char *>(workspace) + kStatusBytes;
    const size_t segs = size_t(a.B) * a.H * (p.n_seg - 1);
    a.n_seg = p.n_seg;
    a.seg_len = p.seg_len;
    a.seg_tot = reinterpret_cast<long long *>(ws);
    a.seg_bad = reinterpret_cast<int *>(ws + tot_bytes(segs));
    a.seg_state = reinterpret_cast<float *>(ws + tot_bytes(segs) + bad_bytes(segs, p));
    a.seg_tiles = p.tiles;
    a.parts = p.parts;
    // Ragged rows by falling length where the blocks are more than the SMs hold at once.
    // Lengths drawn evenly: bf16 B8 L1017 H32 d64 47.6 -> 38.7 us, B16 L2048 H16 d128
    // 146 -> 140, B64 L1024 H4 d64 47.0 -> 42.6, but B32 L500 H8 d128 61.8 -> 63.0; fp32
    // B64 L500 H8 d64 167 -> 109, B32 L300 H32 d128 353 -> 294.  Blocks that all run at
    // once are slower so, with the long ones side by side on the same SMs (fp32 B16
    // L1024 H16 d128 392 -> 428, 386 -> 476 with lengths that rise along the batch).
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    const int64_t at_once = int64_t(sms) * (p.path == 1 ? 1 : a.dk <= 64 ? 8 : a.dk <= 128 ? 4 : 3);
    a.by_length = a.lens != nullptr && a.B > 1 && a.B <= kOrderRows && p.blocks > at_once;
    a.o_part = a.seg_state + segs * a.dv * a.dk;
    const StatusRef st = call_status(workspace);
    if (p.path == 1) return decay_tensor_launch(a, st, stream);
    return io == LR_BF16 ? decay_general_launch<__nv_bfloat16>(a, p, st, stream)
                         : decay_general_launch<float>(a, p, st, stream);
}

}  // namespace lr
