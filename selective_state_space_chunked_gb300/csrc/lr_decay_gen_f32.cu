// lr_decay_gen_f32.cu -- decayed linear attention on the CUDA cores, fp32 I/O,
// and the row and step counts of its configurations
#include "lr_decay_general.cuh"

namespace lr {
template int decay_general_launch<float, false>(const DecayArgs &, const DecayPlan &, StatusRef, cudaStream_t);

namespace {
template <int DKP>
int rows_of(int thread_rows) {
    return thread_rows == 1 ? DecCfg<DKP, 1>::RB : thread_rows == 2 ? DecCfg<DKP, 2>::RB : DecCfg<DKP, 4>::RB;
}
}  // namespace

int decay_general_rows(int64_t dk, int thread_rows) {
    if (dk <= 32) return rows_of<32>(thread_rows);
    if (dk <= 64) return rows_of<64>(thread_rows);
    if (dk <= 128) return rows_of<128>(thread_rows);
    if (dk <= 256) return rows_of<256>(thread_rows);
    return rows_of<512>(thread_rows);
}
}  // namespace lr
