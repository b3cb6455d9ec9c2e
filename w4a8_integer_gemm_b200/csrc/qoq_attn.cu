// qoq_attn.cu -- attention of new tokens over the paged cache: which kernel
// takes which sequence.
//
// A sequence has n_b * G rows per KV head.  Up to kFewRows of them go to the
// kernel that streams the cache through warp-level MMAs, sixteen rows a pass
// (qoq_attn_rows.cu, whose floor is the cache's bytes); more go to the tensor-core
// tiles (qoq_attn_tile.cu).  32 sequences of 2000 tokens, 8 KV heads of 128
// in 4 bits, us: 16 rows 45 against 77 in tiles, 32 rows 67 against 81 (no
// other lengths, widths or bits were swept).
// Each kernel looks at the lengths on the device and skips the other's
// sequences, so a mixed batch takes both launches and no length is read on
// the host.  The caller's max_new saves a launch, and a decode step's rows
// their second column block: 64 sequences of 4000 tokens, groups of 4, 78 us
// with it and 114 without.
#include <algorithm>
#include <atomic>

#include "qoq_attn_internal.h"

namespace qoq {

namespace {

constexpr int kFewRows = 32;
constexpr int kAnyRows = 1 << 30;

struct Plan {
    bool rows, tiles;   // which kernels run
    int few;            // sequences with at most this many rows are the first one's
    size_t rows_bytes, tiles_bytes;
};

Plan plan(int T, int Hq, int Hkv, int d, int max_new)
{
    const int G = Hq / Hkv;
    const int64_t most = (int64_t)std::min(max_new, T) * G;      // rows of a sequence, as far as the caller knows
    Plan p;
    p.rows = G <= kFewRows;
    p.tiles = most > kFewRows;
    p.few = !p.rows ? 0 : p.tiles ? kFewRows : kAnyRows;
    p.rows_bytes = p.rows ? (rows_workspace(d) + 15) & ~(size_t)15 : 0;
    p.tiles_bytes = p.tiles ? tiles_workspace(d) : 0;
    return p;
}

}  // namespace

int attn_sms()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

bool paged_attention_fits(int T, int B, int Hq, int Hkv, int table_pages, int page_size)
{
    return tiles_fit(row_tiles(T, B, Hq / Hkv, 0), Hkv, table_pages, page_size);
}

size_t paged_attention_workspace(int T, int Hq, int Hkv, int d, int max_new)
{
    const Plan p = plan(T, Hq, Hkv, d, max_new);
    return p.rows_bytes + p.tiles_bytes;
}

cudaError_t launch_paged_attention(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                                   const AttnBatch &a, int max_new, float scale, uint16_t *out, int64_t ldo,
                                   void *workspace, cudaStream_t stream)
{
    const Plan p = plan(T, Hq, Hkv, d, max_new);
    void *tiles_ws = reinterpret_cast<uint8_t *>(workspace) + p.rows_bytes;
    // rows in one column block of the MMAs instead of two: 49 us against 62 for 32 sequences of 4000 tokens
    const bool eight = (int64_t)std::min(max_new, T) * (Hq / Hkv) <= 8;
    auto rows = [&](bool join) {
        return launch_paged_rows(q, ldq, T, Hq, Hkv, d, c, a, p.few, eight, scale, out, ldo, workspace, stream, join);
    };
    auto tiles = [&](bool join) {
        return launch_paged_tiles(q, ldq, T, Hq, Hkv, d, c, a, p.few, scale, out, ldo, tiles_ws, stream, p.rows, join);
    };
    // The tiles take over the SMs as the rows' CTAs end, and the joins come last (a mixed batch: 72 us against 73 one
    // after another).
    cudaError_t e = cudaSuccess;
    if (p.rows) e = rows(false);
    if (p.tiles && e == cudaSuccess) e = tiles(false);
    if (p.rows && e == cudaSuccess) e = rows(true);
    if (p.tiles && e == cudaSuccess) e = tiles(true);
    return e;
}

}  // namespace qoq
