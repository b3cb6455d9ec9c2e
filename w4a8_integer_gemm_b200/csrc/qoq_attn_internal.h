// qoq_attn_internal.h -- what the attention operators share on host and
// device: the batch description, the cache, and the launchers behind
// include/qoq_attn.h.  Arguments have been validated by qoq_attn_api.cu.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace qoq {

// The batch: which rows belong to which sequence, and where their tokens are.
struct AttnBatch {
    const int32_t *cu;       // [B + 1]
    const int32_t *kv_len;   // [B]; null for prompts
    const int32_t *table;    // [B][table_pages]; null for prompts
    int B, table_pages, page_size, pages;
    int page_shift;          // page_size == 1 << page_shift
};

struct AttnCache {
    uint8_t *k_codes, *v_codes;
    uint16_t *k_par, *v_par;
    int bits;
};

struct AttnRotary {
    const double *freq;      // radians per position [rot / 2]
    int rot, interleaved;
    float amplitude;
};

// A row of T: its sequence, or -1.
__device__ __forceinline__ int sequence_of(const int32_t *__restrict__ cu, int B, int t)
{
    int lo = 0, hi = B + 1;            // the number of entries <= t lies in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid + 1;
        else hi = mid;
    }
    const int b = lo - 1;
    if (b < 0 || b >= B || t >= __ldg(cu + b + 1)) return -1;
    return b;
}

// The page of position `pos` of sequence b, or -1 (absent).
__device__ __forceinline__ int page_of(const AttnBatch &a, int b, int pos)
{
    if (pos < 0) return -1;
    const int p = pos >> a.page_shift;
    if (p >= a.table_pages) return -1;
    const int page = __ldg(a.table + (size_t)b * a.table_pages + p);
    return page >= 0 && page < a.pages ? page : -1;
}

cudaError_t launch_rotary(const uint16_t *x, int64_t ldx, const int32_t *pos, const AttnRotary &r, int T, int H, int d,
                          uint16_t *y, int64_t ldy, cudaStream_t stream);
cudaError_t launch_cache_append(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const uint16_t *q,
                                int64_t ldq, uint16_t *q_out, int64_t ldqo, int T, int Hq, int Hkv, int d,
                                const AttnRotary &r, const AttnCache &c, const AttnBatch &a, cudaStream_t stream);
cudaError_t launch_cache_read(const AttnCache &c, const AttnBatch &a, int T, int Hkv, int d, uint16_t *K, uint16_t *V,
                              cudaStream_t stream);

// Whether the work of such a call can be counted in 31 bits.
bool paged_attention_fits(int T, int B, int Hq, int Hkv, int table_pages, int page_size);
size_t paged_attention_workspace(int T, int Hq, int Hkv, int d, int max_new);
cudaError_t launch_paged_attention(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                                   const AttnBatch &a, int max_new, float scale, uint16_t *out, int64_t ldo,
                                   void *workspace, cudaStream_t stream);
// SMs of the current device, looked up once per device.
int attn_sms();
// Row tiles that a batch can have at most (sequences with more than `few` rows), and whether their key tiles can be
// counted in 31 bits.
int64_t row_tiles(int T, int B, int G, int few);
bool tiles_fit(int64_t tiles, int Hkv, int table_pages, int page_size);
// Launches `kernel` so that it may start as soon as every CTA of the stream's last kernel allows it (early), or after it.
template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, bool early, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Row tiles on the tensor cores (qoq_attn_tile.cu) for the sequences with more than `few` rows: the work, or (join) the
// joining of its parts.  early: the stream's last kernel is the other sequences', beside which the work may run.
size_t tiles_workspace(int d);
cudaError_t launch_paged_tiles(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                               const AttnBatch &a, int few, float scale, uint16_t *out, int64_t ldo, void *workspace,
                               cudaStream_t stream, bool early, bool join);
// Few rows (qoq_attn_rows.cu): the sequences with at most `few` rows, 8 rows (eight) or 16 to a pass over the cache; the
// work, or the joining of its parts.
size_t rows_workspace(int d);
cudaError_t launch_paged_rows(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                              const AttnBatch &a, int few, bool eight, float scale, uint16_t *out, int64_t ldo,
                              void *workspace, cudaStream_t stream, bool join);
// The tile kernel's error flag (a bounded wait ran out), read and cleared.
cudaError_t read_and_clear_tile_error(int *value);
cudaError_t launch_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                                    int64_t ldv, int T, int Hq, int Hkv, int d, const AttnBatch &a, float scale,
                                    uint16_t *out, int64_t ldo, cudaStream_t stream);

}  // namespace qoq
