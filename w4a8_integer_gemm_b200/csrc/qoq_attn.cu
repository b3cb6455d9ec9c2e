// qoq_attn.cu -- attention of new tokens over the paged cache: which kernel
// takes which sequence.
#include "qoq_attn_internal.h"

namespace qoq {

size_t paged_attention_workspace(int, int, int, int, int, int, int, int)
{
    return 16;
}

cudaError_t launch_paged_attention(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                                   const AttnBatch &a, int, float scale, uint16_t *out, int64_t ldo, void *,
                                   cudaStream_t stream)
{
    return launch_paged_tiles(q, ldq, T, Hq, Hkv, d, c, a, 0, 1, scale, out, ldo, nullptr, stream);
}

}  // namespace qoq
