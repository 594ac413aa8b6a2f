// lr_decay_tensor.cu -- decayed linear attention on the tensor cores
#include "lr_decay_tensor.cuh"

namespace lr {
template int decay_tensor_launch<false>(const DecayArgs &, StatusRef, cudaStream_t);
}
