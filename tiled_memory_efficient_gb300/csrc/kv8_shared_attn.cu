// kv8_shared_attn.cu -- the cache's attention over what sequences see behind a shared prefix.
#include "kv8_attn.cuh"

namespace tme {

int attn_launch_shared(const AttnParams& p, const void* k_pages, const void* v_pages, int D, int page, bool bf16,
                       cudaStream_t stream) {
    return launch_attention<true>(p, k_pages, v_pages, D, page, bf16, stream) == cudaSuccess ? ATTN_OK
                                                                                             : ATTN_ERR_CUDA;
}

}  // namespace tme
