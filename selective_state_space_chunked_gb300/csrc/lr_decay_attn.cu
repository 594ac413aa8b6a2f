// lr_decay_attn.cu -- plan and dispatch of the decayed linear attention.
#include "lr_decay.cuh"

namespace lr {

namespace {
// CUDA-core kernel: the shortest segment, and costs in units of a step of a
// block: a block's start, one segment's state read by a later one, and the
// second launch.  Chosen on sweeps of the segment count over 20 shapes.  fp32
// H16 d128, B2 L2048: 4 segments 263 us, 7 232, 9 (chosen) 202, 12 245; B4 L4096: 1
// 1060, 4 726, 9 (chosen) 668, 14 681; B1 L32768: 9 1791, 19 (chosen) 1267, 24 1484;
// few heads: B1 L8192 H1 d128 32 116, 64 (chosen) 73.5, 96 93; B1 L4096 H2 d64 32
// 48.6, 41 (chosen) 48.6, 45 59, 64 50.
// Blocks with one or two state rows a thread, where four would leave the SMs with few
// blocks.  A step's time in us, costs in steps; kWideUnit: the unit in us of the
// four-row form's costs.  Fitted to sweeps of the rows and the segment count over 39
// shapes; us with the four-row form's plan (and one row where a call had one segment and
// few blocks), and with this: selective scan with heads, fp32, B2 L700 H12 P80 N96 93,
// 50.5 (2 rows, 5 segments); B1 L300 H8 P64 N64 37, 13 (1, 6); B8 L500 H16 P64 N128
// 193, 102 (2, 1); B8 L1017 H32 P64 N64 469, 260 (2, 1); B32 L100 H16 P64 N64 73, 66;
// decayed attention, fp32, B1 L300 H8 d64 28, 12.5; B1 L8192 H1 d128 73.5, 62; B16
// L512 H16 dk64 dv128 219, 219 (4, 1; two rows 193); bf16 B1 L40 H16 d128 9.5, 7.4.
// Of 55 shapes none got more than 1 % slower.
constexpr int64_t kGenMinSeg = 64;
constexpr double kGenBlockCost = 40.0, kGenStateCost = 3.0, kGenLaunchCost = 50.0;
constexpr int64_t kGenMaxSeg = 96;
constexpr double kWideUnit = 0.115, kWideUnitNarrowKeys = 0.09;
constexpr int64_t kFewMinSeg = 48;
constexpr double kFewBlockCost = 15.0, kFewStateCost = 4.0, kFewLaunchTime = 3.0, kFewMargin = 1.05;
// Tensor-core kernel: the shortest sequence it takes (bf16, on it and on the CUDA
// cores: B1 L48 H4 d128 9.6 and 10.9 us, L32 9.7 and 8.1; B4 L48 H32 d64 10.8 and
// 11.4; B1 H8 dk256, L48 12.0 and 15.2, L32 12.0 and 10.8; the other way, B8 L48 H16
// d128 21.4 and 19.1), and costs in units of a chunk's time: a chunk of the first
// launch, a block's start, and one segment's state read by a later one.  Against
// sweeps of the segment count over 11 shapes the plan's choice is the best or
// within 4 %: B1 L32768 H16 d128 1 segment 571 us, 2 433, 4 (chosen) 234, 8 274;
// B1 L16384 H8 dk64 6 81, 9 60, 12 50.5, 16 (chosen) 47.0, 19 45.4, 24 68; B4 L2048
// H16 1 (chosen) 48.4, 2 76.
// The scan with heads takes the same costs, though its chunks are longer and a chunk of its
// first launch is 0.37 of one of the last (70 us of 190 at B1 L32768 H16 P128 N128).
constexpr int64_t kMaxSeg = 32;
constexpr int64_t kTensorMinLen = 48;
constexpr double kFirstCost = 0.6, kBlockCost = 3.0, kStateCost = 1.0;
}  // namespace

namespace {
size_t tot_bytes(size_t segs) { return (segs * sizeof(long long) + 15) / 16 * 16; }
// a scan's gates: per step a weight, a readout factor, one to the segment's end and
// two of its own; per chunk a record; per segment what is left
size_t gate_bytes(size_t bh, int64_t L, int n_seg) {
    const size_t chunks = bh * size_t((L + kDecayChunk - 1) / kDecayChunk);
    return chunks * (kDecayChunk * 5 * sizeof(float) + kChunkRecord) + (bh * n_seg * sizeof(float) + 15) / 16 * 16;
}
size_t bad_bytes(size_t segs, const DecayPlan &p) { return (segs * p.tiles * sizeof(int) + 15) / 16 * 16; }
}  // namespace

int decay_plan(int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv, lr_dtype io, bool heads,
               DecayPlan *p) {
    (void)Hk;
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    int64_t n = 1, unit = 16;
    p->thread_rows = 4;
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
        const int64_t rows = decay_general_rows(dk, 4), threads = dk <= 64 ? 64 : 128, slots = dk <= 128 ? 4 : 3;
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
        // fewer rows a thread: from the time of a step (us) with one block on the
        // fullest SM to that with as many as it holds
        struct Step {
            double one, full;
        };
        static constexpr Step kSteps[3][2] = {{{0.07, 0.09}, {0.08, 0.125}},     // to 64 keys: one row, two
                                              {{0.095, 0.175}, {0.154, 0.2}},    // to 128
                                              {{0.1, 0.2}, {0.15, 0.24}}};       // to 256
        best *= dk <= 64 ? kWideUnitNarrowKeys : kWideUnit;
        for (int r = 1; r <= 2 && dk <= (io == LR_BF16 ? 128 : 256); ++r) {
            const Step &st = kSteps[dk <= 64 ? 0 : dk <= 128 ? 1 : 2][r - 1];
            const int64_t few_rows = decay_general_rows(dk, r), few = B * H * ((dv + few_rows - 1) / few_rows);
            auto step_time = [&](int64_t b) {   // of all rounds of blocks
                const int64_t most = (b + sms - 1) / sms, full = most / slots, rest = most % slots;
                const double last = rest == 0 ? 0.0 : st.one + (st.full - st.one) * double(rest - 1) / double(slots - 1);
                return double(full) * st.full + (full > 0 ? 0.84 : 1.0) * last;
            };
            for (int64_t s = 1; s == 1 || (s <= kGenMaxSeg && s * kFewMinSeg <= L); ++s) {
                const double per = double(((L + s - 1) / s + unit - 1) / unit * unit);
                double t = step_time(few * s) * (per + kFewBlockCost + kFewStateCost * double(s));
                if (s > 1) t += step_time(few * (s - 1)) * (0.36 * per + kFewBlockCost) + kFewLaunchTime;
                if (kFewMargin * t < best) best = kFewMargin * t, n = s, p->thread_rows = r;
            }
        }
    }
    p->seg_len = ((L + n - 1) / n + unit - 1) / unit * unit;
    p->n_seg = int((L + p->seg_len - 1) / p->seg_len);
    const int64_t rows = p->path == 1 ? kDecayRows : decay_general_rows(dk, p->thread_rows);
    p->tiles = int((dv + rows - 1) / rows) * p->parts;
    p->blocks = B * H * p->tiles * p->n_seg;
    const size_t segs = size_t(B) * H * (p->n_seg - 1);
    p->ws_bytes = kStatusBytes + tot_bytes(segs) + bad_bytes(segs, *p) + segs * dv * dk * sizeof(float);
    if (p->parts > 1) p->ws_bytes += size_t(p->parts) * B * L * H * dv * sizeof(float);
    if (heads && p->path == 1) p->ws_bytes = (p->ws_bytes + 15) / 16 * 16 + gate_bytes(B * H, L, p->n_seg);
    return LR_OK;
}

int decay_attn_launch(DecayArgs a, lr_dtype io, const DecayPlan &p, bool heads, void *workspace, cudaStream_t stream) {
    unsigned char *ws = static_cast<unsigned char *>(workspace) + kStatusBytes;
    const size_t segs = size_t(a.B) * a.H * (p.n_seg - 1);
    a.n_seg = p.n_seg;
    a.seg_len = p.seg_len;
    a.seg_tot = reinterpret_cast<long long *>(ws);
    a.seg_bad = reinterpret_cast<int *>(ws + tot_bytes(segs));
    a.seg_state = reinterpret_cast<float *>(ws + tot_bytes(segs) + bad_bytes(segs, p));
    a.seg_tiles = p.tiles;
    a.parts = p.parts;
    // Ragged rows by falling length, lengths drawn evenly (us in the batch's order, by
    // length).  Tensor cores, more blocks than SMs: bf16 B8 L1017 H32 d64 47.6, 38.7;
    // B16 L2048 H16 d128 146, 140; B64 L1024 H4 d64 47.0, 42.6; but B32 L500 H8 d128
    // 61.8, 63.0.  CUDA cores, more than four blocks per SM: fp32 B64 L500 H8 d64 (6.7)
    // 167, 109; B32 L300 H32 d128 (13.5) 353, 294.  With fewer, the long rows stand
    // beside one another on some SMs: B16 L1024 H16 d128 (3.4) 392, 428, and 386, 476
    // with lengths that rise along the batch; B8 L1017 H32 d64 (3.4) 175, 179.
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    a.by_length = a.lens != nullptr && a.B > 1 && a.B <= kOrderRows && p.blocks > (p.path == 1 ? 1 : 4) * sms;
    a.o_part = a.seg_state + segs * a.dv * a.dk;
    const StatusRef st = call_status(workspace);
    if (heads) {
        if (p.path == 1) {
            const size_t bh = size_t(a.B) * a.H, chunks = bh * size_t((a.L + kDecayChunk - 1) / kDecayChunk);
            const size_t steps = chunks * kDecayChunk;
            unsigned char *g = static_cast<unsigned char *>(workspace) + p.ws_bytes - gate_bytes(bh, a.L, p.n_seg);
            a.hd.chunk = g;
            a.hd.weight = reinterpret_cast<float *>(g + chunks * kChunkRecord);
            a.hd.readout = a.hd.weight + steps;
            a.hd.to_end = a.hd.readout + steps;
            a.hd.own = reinterpret_cast<float2 *>(a.hd.to_end + steps);
            a.hd.left = reinterpret_cast<float *>(a.hd.own + steps);
            return heads_tensor_launch(a, st, stream);
        }
        return io == LR_BF16 ? decay_general_launch<__nv_bfloat16, true>(a, p, st, stream)
                             : decay_general_launch<float, true>(a, p, st, stream);
    }
    if (p.path == 1) return decay_tensor_launch(a, st, stream);
    return io == LR_BF16 ? decay_general_launch<__nv_bfloat16, false>(a, p, st, stream)
                         : decay_general_launch<float, false>(a, p, st, stream);
}

}  // namespace lr
