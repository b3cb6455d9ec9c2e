// qoq_attn_api.cu -- the extern "C" entry points declared in
// include/qoq_attn.h: argument validation on the host, then the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/qoq_attn.h"
#include "qoq_attn_internal.h"
#include "qoq_internal.h"

namespace {

using qoq::aligned16;
using qoq::check_device;

constexpr int kMaxRows = 1 << 21;
constexpr int kMaxSequences = 1 << 16;
constexpr int kMaxHeads = 1024;
constexpr int kMaxGroup = 64;
constexpr int kMaxTokens = 1 << 24;      // positions of one sequence the table can hold

bool aligned4(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

int from_cuda(cudaError_t e)
{
    return e == cudaSuccess ? QOQ_OK : QOQ_ERR_CUDA;
}

// A matrix of heads [T][H][d] with row stride ld.
bool valid_rows(const void *x, int64_t ld, int H, int d)
{
    return x && aligned16(x) && ld >= (int64_t)H * d && ld % 8 == 0;
}

bool valid_counts(int T, int B)
{
    return T >= 0 && T <= kMaxRows && B >= 0 && B <= kMaxSequences;
}

bool valid_heads(int Hq, int Hkv, int d)
{
    return Hkv >= 1 && Hq >= Hkv && Hq <= kMaxHeads && Hq % Hkv == 0 && Hq / Hkv <= kMaxGroup && (d == 64 || d == 128);
}

bool valid_paging(int page_size, int pages, int table_pages)
{
    return (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128) && pages >= 1 &&
           table_pages >= 1 && (int64_t)table_pages * page_size <= kMaxTokens;
}

int page_shift(int page_size)
{
    return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
}

bool valid_rotary(const double *freq, int d, int rot, int interleaved, float amplitude)
{
    if (rot < 0 || rot > d || rot % 16 != 0 || (interleaved != 0 && interleaved != 1)) return false;
    return rot == 0 || (freq && aligned16(freq) && std::isfinite(amplitude));
}

bool valid_cache(const void *kc, const void *vc, const void *kp, const void *vp, int bits)
{
    return (bits == 4 || bits == 8) && kc && vc && kp && vp && aligned16(kc) && aligned16(vc) && aligned16(kp) &&
           aligned16(vp);
}

bool valid_index(const void *p)
{
    return p && aligned4(p);
}

}  // namespace

extern "C" {

int qattn_rotary(const uint16_t *x, int64_t ldx, const int32_t *pos, const double *freq, int T, int H, int d, int rot,
                 int interleaved, float amplitude, uint16_t *y, int64_t ldy, void *stream)
{
    if (T < 0 || T > kMaxRows || H < 1 || H > kMaxHeads || d < 16 || d > 512 || d % 16 != 0) return QOQ_ERR_INVALID_ARG;
    if (!valid_rotary(freq, d, rot, interleaved, amplitude)) return QOQ_ERR_INVALID_ARG;
    if (T == 0) return QOQ_OK;
    if (!valid_rows(x, ldx, H, d) || !valid_rows(y, ldy, H, d) || !valid_index(pos)) return QOQ_ERR_INVALID_ARG;
    const int dev = check_device();
    if (dev != QOQ_OK) return dev;
    return from_cuda(
        qoq::launch_rotary(x, ldx, pos, {freq, rot, interleaved, amplitude}, T, H, d, y, ldy, (cudaStream_t)stream));
}

int qattn_cache_append(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const uint16_t *q, int64_t ldq,
                       uint16_t *q_out, int64_t ldqo, int T, int Hq, int Hkv, int d, const double *freq, int rot,
                       int interleaved, float amplitude, int bits, int page_size, int pages, uint8_t *k_codes,
                       uint8_t *v_codes, uint16_t *k_par, uint16_t *v_par, const int32_t *table, int table_pages,
                       const int32_t *cu, const int32_t *kv_len, int B, void *stream)
{
    if (!valid_counts(T, B) || !valid_heads(q ? Hq : Hkv, Hkv, d) || !valid_paging(page_size, pages, table_pages) ||
        !valid_rotary(freq, d, rot, interleaved, amplitude) || (q && rot == 0))
        return QOQ_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return QOQ_OK;
    if (!valid_rows(k, ldk, Hkv, d) || !valid_rows(v, ldv, Hkv, d) ||
        !valid_cache(k_codes, v_codes, k_par, v_par, bits) || !valid_index(table) || !valid_index(cu) ||
        !valid_index(kv_len))
        return QOQ_ERR_INVALID_ARG;
    if (q && (!valid_rows(q, ldq, Hq, d) || !valid_rows(q_out, ldqo, Hq, d))) return QOQ_ERR_INVALID_ARG;
    const int dev = check_device();
    if (dev != QOQ_OK) return dev;
    return from_cuda(qoq::launch_cache_append(k, ldk, v, ldv, q, ldq, q_out, ldqo, T, q ? Hq : 0, Hkv, d,
                                              {freq, rot, interleaved, amplitude},
                                              {k_codes, v_codes, k_par, v_par, bits},
                                              {cu, kv_len, table, B, table_pages, page_size, pages, page_shift(page_size)},
                                              (cudaStream_t)stream));
}

int qattn_cache_read(const uint8_t *k_codes, const uint8_t *v_codes, const uint16_t *k_par, const uint16_t *v_par,
                     int bits, int page_size, int pages, int Hkv, int d, const int32_t *table, int table_pages,
                     const int32_t *cu, const int32_t *kv_len, int B, int T, uint16_t *K, uint16_t *V, void *stream)
{
    if (!valid_counts(T, B) || !valid_heads(Hkv, Hkv, d) || !valid_paging(page_size, pages, table_pages))
        return QOQ_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return QOQ_OK;
    if (!valid_cache(k_codes, v_codes, k_par, v_par, bits) || !valid_index(table) || !valid_index(cu) ||
        !valid_index(kv_len) || !K || !V || !aligned16(K) || !aligned16(V))
        return QOQ_ERR_INVALID_ARG;
    const int dev = check_device();
    if (dev != QOQ_OK) return dev;
    return from_cuda(qoq::launch_cache_read(
        {const_cast<uint8_t *>(k_codes), const_cast<uint8_t *>(v_codes), const_cast<uint16_t *>(k_par),
         const_cast<uint16_t *>(v_par), bits},
        {cu, kv_len, table, B, table_pages, page_size, pages, page_shift(page_size)}, T, Hkv, d, K, V, (cudaStream_t)stream));
}

size_t qattn_paged_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int d, int table_pages, int page_size,
                                             int max_new)
{
    if (!valid_counts(T, B) || !valid_heads(Hq, Hkv, d) || !valid_paging(page_size, 1, table_pages) || max_new < 1)
        return 0;
    if (T == 0 || B == 0 || !qoq::paged_attention_fits(T, B, Hq, Hkv, table_pages, page_size)) return 0;
    return qoq::paged_attention_workspace(T, Hq, Hkv, d, max_new);
}

int qattn_paged_attention(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const uint8_t *k_codes,
                          const uint8_t *v_codes, const uint16_t *k_par, const uint16_t *v_par, int bits,
                          int page_size, int pages, const int32_t *table, int table_pages, const int32_t *cu,
                          const int32_t *kv_len, int B, int max_new, float scale, uint16_t *out, int64_t ldo,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    if (!valid_counts(T, B) || !valid_heads(Hq, Hkv, d) || !valid_paging(page_size, pages, table_pages) ||
        max_new < 1 || !std::isfinite(scale))
        return QOQ_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return QOQ_OK;
    if (!qoq::paged_attention_fits(T, B, Hq, Hkv, table_pages, page_size)) return QOQ_ERR_INVALID_ARG;
    if (!valid_rows(q, ldq, Hq, d) || !valid_rows(out, ldo, Hq, d) ||
        !valid_cache(k_codes, v_codes, k_par, v_par, bits) || !valid_index(table) || !valid_index(cu) ||
        !valid_index(kv_len))
        return QOQ_ERR_INVALID_ARG;
    const size_t need = qoq::paged_attention_workspace(T, Hq, Hkv, d, max_new);
    if (workspace_bytes < need || (need && (!workspace || !aligned16(workspace)))) return QOQ_ERR_INVALID_ARG;
    const int dev = check_device();
    if (dev != QOQ_OK) return dev;
    return from_cuda(qoq::launch_paged_attention(
        q, ldq, T, Hq, Hkv, d,
        {const_cast<uint8_t *>(k_codes), const_cast<uint8_t *>(v_codes), const_cast<uint16_t *>(k_par),
         const_cast<uint16_t *>(v_par), bits},
        {cu, kv_len, table, B, table_pages, page_size, pages, page_shift(page_size)}, max_new, scale, out, ldo, workspace,
        (cudaStream_t)stream));
}

int qattn_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                           int64_t ldv, int T, int Hq, int Hkv, int d, const int32_t *cu, int B, float scale,
                           uint16_t *out, int64_t ldo, void *stream)
{
    if (!valid_counts(T, B) || !valid_heads(Hq, Hkv, d) || !std::isfinite(scale)) return QOQ_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return QOQ_OK;
    if (!valid_rows(q, ldq, Hq, d) || !valid_rows(k, ldk, Hkv, d) || !valid_rows(v, ldv, Hkv, d) ||
        !valid_rows(out, ldo, Hq, d) || !valid_index(cu))
        return QOQ_ERR_INVALID_ARG;
    const int dev = check_device();
    if (dev != QOQ_OK) return dev;
    return from_cuda(qoq::launch_prompt_attention(q, ldq, k, ldk, v, ldv, T, Hq, Hkv, d,
                                                  {cu, nullptr, nullptr, B, 0, 0, 0, 0}, scale, out, ldo,
                                                  (cudaStream_t)stream));
}

}  // extern "C"
