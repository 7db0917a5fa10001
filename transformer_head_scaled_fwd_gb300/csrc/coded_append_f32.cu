// coded_append_f32.cu -- the same for fp32 tensors: the two files are compiled side by side.
#include "coded_append.cuh"

namespace mha {

cudaError_t launch_coded_append_f32(const CodedAppendParams& p, cudaStream_t s) { return launch_t<float>(p, s); }

}  // namespace mha
