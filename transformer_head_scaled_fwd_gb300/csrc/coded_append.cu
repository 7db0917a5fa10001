// coded_append.cu -- launches of the append to a cache in 8 bits (coded_append.cuh): bf16 tensors, and which type theirs is.
#include "coded_append.cuh"

namespace mha {

cudaError_t launch_coded_append(const CodedAppendParams& p, bool bf16, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_coded_append_f32(p, s);
}

}  // namespace mha
