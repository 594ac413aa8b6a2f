// lr_decay_gen_f32.cu -- decayed linear attention on the CUDA cores, fp32 I/O,
// and the row and step counts of its configurations
#include "lr_decay_general.cuh"

namespace lr {
template int decay_general_launch<float>(const DecayArgs &, const DecayPlan &, StatusRef, cudaStream_t);

namespace {
template <int DKP>
int rows_of(bool narrow) {
    return narrow ? DecCfg<DKP, true>::RB : DecCfg<DKP, false>::RB;
}
}  // namespace

int decay_general_rows(int64_t dk, bool narrow) {
    if (dk <= 32) return rows_of<32>(narrow);
    if (dk <= 64) return rows_of<64>(narrow);
    if (dk <= 128) return rows_of<128>(narrow);
    if (dk <= 256) return rows_of<256>(narrow);
    return rows_of<512>(narrow);
}
}  // namespace lr
