// lr_heads_tensor.cu -- selective scan with heads on the tensor cores
#include "lr_decay_tensor.cuh"

namespace lr {
template int decay_tensor_launch<true>(const DecayArgs &, StatusRef, cudaStream_t);
}
