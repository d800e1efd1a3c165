// attention_fwd_pages.cu -- the attention forward over a paged cache, for more query rows than
// attention_paged.cu takes (see attention_fwd.cuh).
#include "attention_fwd.cuh"

namespace uly {

cudaError_t attn_fwd_pages_launch(const AttnFwdArgs& a, cudaStream_t stream, int device, int64_t cap,
                                  int sm_count)
{
    return af_launch_types<kAfLong, true, true>(a, stream, device, cap, sm_count);
}

cudaError_t attn_fwd_pages_status(unsigned* status, bool clear) { return af_status(status, clear); }

}  // namespace uly
