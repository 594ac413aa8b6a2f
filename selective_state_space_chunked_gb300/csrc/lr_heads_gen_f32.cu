// lr_heads_gen_f32.cu -- selective scan with heads on the CUDA cores, fp32 I/O
#include "lr_decay_general.cuh"

namespace lr {
template int decay_general_launch<float, true>(const DecayArgs &, const DecayPlan &, StatusRef, cudaStream_t);
}
