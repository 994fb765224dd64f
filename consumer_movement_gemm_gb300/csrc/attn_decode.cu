// attn_decode.cu -- attention of one new token over a bf16 cache, and what both
// cache types share on the host (attn_decode.cuh has the kernel).
#include "attn_decode.cuh"

namespace tovl {

AttnShape attn_decode_shape(int dim, bool e4m3, int group, bool pair)
{
    const auto shape = [](auto s) {
        using S = decltype(s);
        return AttnShape{S::kTile, S::kBlockRow, S::kWarps, S::kHeads, S::kPart};
    };
    return e4m3 ? attn::with_shape<true>(dim, group, pair, shape) : attn::with_shape<false>(dim, group, pair, shape);
}

bool attn_decode_pairs(int dim, bool e4m3, int group) { return dim > 128 && !e4m3 && (group + 7) / 8 % 2 == 0; }

int attn_decode_together(const AttnShape& s, int heads, int dim, bool e4m3)
{
    const int row = dim * (e4m3 ? 1 : 2);
    int n = 1;
    while (n < 8 && n * row % 128 && heads % (2 * n) == 0 && s.warps % (2 * n) == 0) n *= 2;
    return n;
}

long long attn_decode_workspace(int heads, int group, int dim, int num_sms)
{
    long long most = 0;
    for (int i = 0; i < 3; ++i) {
        const bool e4m3 = i == 1, pair = i == 2;
        if (pair && !attn_decode_pairs(dim, e4m3, group)) continue;
        const AttnShape s = attn_decode_shape(dim, e4m3, group, pair);
        // of each warp, of each CTA and of each group of CTAs, two of a head
        const int together = pair ? 2 : attn_decode_together(s, heads, dim, e4m3);
        const long long bytes = 4LL * s.part * num_sms * (s.warps + 4 * together);
        if (bytes > most) most = bytes;
    }
    return most;
}

cudaError_t prepare_attn_decode()
{
    const cudaError_t e = attn::prepare<false>();
    return e != cudaSuccess ? e : prepare_attn_decode_e4m3();
}

cudaError_t launch_attn_decode(const AttnParams& p, bool e4m3, int num_sms, cudaStream_t stream, bool pdl)
{
    return e4m3 ? launch_attn_decode_e4m3(p, num_sms, stream, pdl) : attn::launch<false>(p, num_sms, stream, pdl);
}

}  // namespace tovl
