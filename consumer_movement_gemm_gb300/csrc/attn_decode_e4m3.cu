// attn_decode_e4m3.cu -- attention of one new token over an e4m3 cache.
#include "attn_decode.cuh"

namespace tovl {

cudaError_t prepare_attn_decode_e4m3() { return attn::prepare<true>(); }

cudaError_t launch_attn_decode_e4m3(const AttnParams& p, int num_sms, cudaStream_t stream, bool pdl)
{
    return attn::launch<true>(p, num_sms, stream, pdl);
}

}  // namespace tovl
