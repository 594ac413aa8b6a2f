// lr_decay_gen_bf16.cu -- decayed linear attention on the CUDA cores, bf16 I/O
// (a translation unit of its own so that the build runs the types in parallel)
#include "lr_decay_general.cuh"

namespace lr {
template int decay_general_launch<__nv_bfloat16, false>(const DecayArgs &, const DecayPlan &, StatusRef, cudaStream_t);
}
