// lr_heads_gen_bf16.cu -- selective scan with heads on the CUDA cores, bf16 I/O
#include "lr_decay_general.cuh"

namespace lr {
template int decay_general_launch<__nv_bfloat16, true>(const DecayArgs &, const DecayPlan &, StatusRef, cudaStream_t);
}
