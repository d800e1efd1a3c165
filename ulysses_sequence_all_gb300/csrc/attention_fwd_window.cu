// attention_fwd_window.cu -- the attention forward with a sliding window (see attention_fwd.cuh).
#include "attention_fwd.cuh"

namespace uly {

// The long layout at every length: 2 x 4,095 tokens, 32 heads over 8, windows of 64, 256, 1,024 and 2,048 keys
// took 67, 74, 119 and 164 us with it, 71, 74, 138 and 201 with the short one. Rows that fit one tile too: 64
// of them on 4 caches of 8,000 keys (8 key heads, window 4,096) 30 us, in two parts of the keys 32.
cudaError_t attn_fwd_window_launch(const AttnFwdArgs& a, cudaStream_t stream, int device, int64_t cap,
                                   int sm_count)
{
    return af_launch_types<kAfLong, true, false>(a, stream, device, cap, sm_count);
}

cudaError_t attn_fwd_window_status(unsigned* status, bool clear) { return af_status(status, clear); }

}  // namespace uly
