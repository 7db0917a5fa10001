// coded_attn_f32.cu -- the same for fp32 queries: the two files are compiled side by side.
#include "coded_attn.cuh"

namespace mha {

cudaError_t launch_coded_attn_f32(const PagedAttnParams& p, bool int8, cudaStream_t s) {
    return int8 ? launch_t<float, true>(p, s) : launch_t<float, false>(p, s);
}

}  // namespace mha
