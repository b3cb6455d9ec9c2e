// qoq_attn.cu -- attention of new tokens over the paged cache: which kernel
// takes which sequence.
//
// A sequence has n_b * G rows per KV head.  Up to kFewRows of them fit one
// pass of the kernel that streams the cache through warp-level MMAs
// (qoq_attn_rows.cu, bound by the cache's bytes); more go to the tensor-core
// tiles (qoq_attn_tile.cu).  Each kernel looks at the lengths on the device
// and skips the other's sequences, so a mixed batch takes both launches and
// no length is read on the host.  The caller's max_new saves a launch.
#include <algorithm>

#include "qoq_attn_internal.h"

namespace qoq {

constexpr int kFewRows = 16;
constexpr int kAnyRows = 1 << 30;

size_t paged_attention_workspace(int, int, int, int, int d, int, int, int)
{
    return rows_workspace(d);
}

cudaError_t launch_paged_attention(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                                   const AttnBatch &a, int max_new, float scale, uint16_t *out, int64_t ldo,
                                   void *workspace, cudaStream_t stream)
{
    const int G = Hq / Hkv;
    const int64_t most = (int64_t)std::min(max_new, T) * G;      // rows of a sequence, as far as the caller knows
    const bool tiles = most > kFewRows;
    if (G <= kFewRows) {
        const cudaError_t e = launch_paged_rows(q, ldq, T, Hq, Hkv, d, c, a, tiles ? kFewRows : kAnyRows, most <= 8,
                                                scale, out, ldo, workspace, stream);
        if (e != cudaSuccess || !tiles) return e;
    }
    return launch_paged_tiles(q, ldq, T, Hq, Hkv, d, c, a, G <= kFewRows ? kFewRows : 0, 1, scale, out, ldo, nullptr,
                              stream);
}

}  // namespace qoq
