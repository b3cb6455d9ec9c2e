// qoq_attn.cu -- attention of new tokens over the paged cache, and causal
// attention of whole prompts: one warp per (row, query head), one pass over
// the keys with the running maximum and sum of the softmax in FP32.  Each
// lane owns D / 32 neighbouring channels; a score is a warp reduction.
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "qoq_attn_internal.h"
#include "qoq_quant.cuh"

namespace qoq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// D / 32 channels of a cached row, as FP32.
template <int D, int BITS>
__device__ __forceinline__ void cached(const uint8_t *codes, const uint16_t *par, size_t row, int lane,
                                       float (&x)[D / 32])
{
    const uint32_t p = __ldg(reinterpret_cast<const uint32_t *>(par) + row);
    const float s = half_bits_to_float((uint16_t)(p & 0xFFFFu)), m = half_bits_to_float((uint16_t)(p >> 16));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const int ch = lane * (D / 32) + i;
        const uint32_t byte = __ldg(codes + row * (D * BITS / 8) + ch * BITS / 8);
        x[i] = fmaf(s, (float)(BITS == 4 ? (byte >> (4 * (ch & 1))) & 15u : byte), m);
    }
}

template <int D>
__device__ __forceinline__ void plain(const uint16_t *row, int lane, float (&x)[D / 32])
{
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = half_bits_to_float(__ldg(row + lane * (D / 32) + i));
}

// BITS 0: prompt (k, v FP16 rows of the batch itself).
template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) attn_row_kernel(const uint16_t *__restrict__ q, int64_t ldq, int T, int Hq,
                                                            int Hkv, const uint16_t *__restrict__ k, int64_t ldk,
                                                            const uint16_t *__restrict__ v, int64_t ldv, AttnCache c,
                                                            AttnBatch a, float scale, uint16_t *__restrict__ out,
                                                            int64_t ldo)
{
    constexpr int N = D / 32;
    const int64_t e = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (e >= (int64_t)T * Hq) return;
    const int t = (int)(e / Hq), h = (int)(e % Hq), hk = h / (Hq / Hkv);
    const int b = sequence_of(a.cu, a.B, t);
    if (b < 0) return;
    const int first = __ldg(a.cu + b), last = __ldg(a.cu + b + 1);
    const int pos = BITS ? __ldg(a.kv_len + b) - (last - t) : t - first;   // of this row; it sees 0 .. pos
    float qf[N], o[N], x[N];
    plain<D>(q + t * ldq + (size_t)h * D, lane, qf);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j <= pos; ++j) {
        size_t row = 0;
        if (BITS) {
            const int page = page_of(a, b, j);
            if (page < 0) continue;
            row = ((size_t)page * Hkv + hk) * a.page_size + j % a.page_size;
            cached<D, BITS ? BITS : 4>(c.k_codes, c.k_par, row, lane, x);
        } else {
            plain<D>(k + (first + j) * ldk + (size_t)hk * D, lane, x);
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) s = fmaf(qf[i], x[i], s);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= scale;
        const float m1 = fmaxf(m, s), keep = expf(m - m1), p = expf(s - m1);
        m = m1;
        l = fmaf(l, keep, p);
        if (BITS) cached<D, BITS ? BITS : 4>(c.v_codes, c.v_par, row, lane, x);
        else plain<D>(v + (first + j) * ldv + (size_t)hk * D, lane, x);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], keep, p * x[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        out[t * ldo + (size_t)h * D + lane * N + i] = float_to_half_bits(l > 0.0f ? o[i] / l : 0.0f);
}

}  // namespace

size_t paged_attention_workspace(int, int, int, int, int, int, int, int)
{
    return 16;
}

cudaError_t launch_paged_attention(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                                   const AttnBatch &a, int, float scale, uint16_t *out, int64_t ldo, void *,
                                   cudaStream_t stream)
{
    const unsigned grid = (unsigned)(((int64_t)T * Hq + kWarps - 1) / kWarps);
    auto run = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, stream>>>(q, ldq, T, Hq, Hkv, nullptr, 0, nullptr, 0, c, a, scale, out, ldo);
    };
    if (d == 128) c.bits == 4 ? run(attn_row_kernel<128, 4>) : run(attn_row_kernel<128, 8>);
    else c.bits == 4 ? run(attn_row_kernel<64, 4>) : run(attn_row_kernel<64, 8>);
    return cudaGetLastError();
}

cudaError_t launch_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                                    int64_t ldv, int T, int Hq, int Hkv, int d, const AttnBatch &a, float scale,
                                    uint16_t *out, int64_t ldo, cudaStream_t stream)
{
    const unsigned grid = (unsigned)(((int64_t)T * Hq + kWarps - 1) / kWarps);
    auto run = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, stream>>>(q, ldq, T, Hq, Hkv, k, ldk, v, ldv, AttnCache{}, a, scale, out, ldo);
    };
    d == 128 ? run(attn_row_kernel<128, 0>) : run(attn_row_kernel<64, 0>);
    return cudaGetLastError();
}

}  // namespace qoq
