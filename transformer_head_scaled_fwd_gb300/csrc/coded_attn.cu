// coded_attn.cu -- launches of attention over a cache in 8 bits (coded_attn.cuh): bf16 queries, and which type's they are.
#include "coded_attn.cuh"

namespace mha {

size_t coded_attn_workspace(int d) { return line_workspace(d, 2); }

cudaError_t launch_coded_attn(const PagedAttnParams& p, bool bf16, bool int8, cudaStream_t s) {
    if (!bf16) return launch_coded_attn_f32(p, int8, s);
    return int8 ? launch_t<__nv_bfloat16, true>(p, s) : launch_t<__nv_bfloat16, false>(p, s);
}

}  // namespace mha
