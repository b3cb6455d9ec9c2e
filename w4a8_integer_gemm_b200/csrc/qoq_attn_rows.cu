// qoq_attn_rows.cu -- attention of few rows (a decode step: one new token,
// the query heads of a KV head) over the paged 4/8-bit cache.
//
// Bound: the cache's bytes, read once.  What has to stay below that is the
// instructions that turn codes into tensor-core operands, so a code is never
// scaled on its own: with x = s c + m per token (c centred: c' = c - off,
// m' = m + off s)
//     score_j = s_j (q . c'_j) + m'_j sum(q)
//     out     = sum_j (p_j s_j) c'_j + sum_j p_j m'_j
// the products run on the raw codes, exact in FP16, and the scales touch one
// number per token.
//
// A warp works alone on its own tokens, without barriers or shared memory:
// the cache's bytes go from global memory straight into the fragments of
// warp-level MMAs (m16n8k16, FP32 sums; the rows as the 8-wide N dimension):
//     S^T[token][row]   = codes of K (A, tokens x channels) x q (B)
//     O^T[channel][row] = codes of V^T (A, channels x tokens) x p s (B)
// Which channel sits at which fragment position does not matter as long as
// q, and O's write-out, agree; so a lane reads 16 neighbouring bytes of a key
// and D/64 * BITS/2 of a value.  The weights go from the layout of S^T to that of B
// by one 8x8 transposition (movmatrix) each.  The next group's loads are issued as
// soon as the registers they fill have been consumed.
//
// Running maximum m, sum l and sum of p m' in FP32; m may lag behind by 2^8,
// so O is rescaled rarely.  The weights p s are rounded to FP16 (half a step
// each); they are scaled by a power of two per row, k, that follows their
// own maximum, so that small scales do not underflow.
//
// Work: items of 256 tokens of a (sequence, row tile, KV head), in that
// order; CTA c of P takes items c I / P .. (c + 1) I / P - 1, so all CTAs
// read the same number of bytes whatever the lengths.  A run of items of one
// (sequence, row tile, head) that lies within a CTA is finished there; one
// that spans CTAs leaves a partial result in each and a second kernel joins
// them, in order.
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "qoq_attn_device.cuh"
#include "qoq_attn_internal.h"
#include "qoq_ptx.cuh"
#include "qoq_quant.cuh"

namespace qoq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kItem = 256;              // tokens of an item
constexpr uint32_t kNone = 0xFFFFFFFFu;

struct RowsArgs {
    const uint16_t *q;
    int64_t ldq, ldo;
    uint16_t *out;
    AttnCache c;
    AttnBatch a;
    int T, Hq, Hkv, G;
    int few;            // sequences with more rows are another kernel's
    float scale_log2;   // scale * log2(e)
    float *part;        // [P][2][rows][D + 2]
    int4 *joined;       // [P]: (sequence or -1, first row, KV head, first CTA) of the run that ends in CTA c's first part
};

// D (16 x 8, FP32) += A (16 x 16, FP16, row) * B (16 x 8, FP16, col).
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (code - off) pairs of a word: 4 bits: nibbles (0, 4) and (1, 5) of the 16-bit halves' low bytes
__device__ __forceinline__ uint32_t pair_lo(uint32_t x)
{
    return sub_h2((x & 0x000F000Fu) | 0x64006400u, 0x64086408u);   // 1024 + c - 1032
}

__device__ __forceinline__ uint32_t pair_hi(uint32_t x)
{
    return sub_h2((x & 0x00F000F0u) | 0x54005400u, 0x54805480u);   // 64 + c - 72
}

// 8 bits: bytes (0, 1) or (2, 3) of x
__device__ __forceinline__ uint32_t bytes_lo(uint32_t x)
{
    return sub_h2(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
}

__device__ __forceinline__ uint32_t bytes_hi(uint32_t x)
{
    return sub_h2(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w)
{
    if (N == 1) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else if (N == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = x.x;
        w[1] = x.y;
    } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
    }
}

template <int D, int BITS, int NT>
struct RowsCfg {
    static constexpr int kRowBytes = D * BITS / 8;
    static constexpr int kKW = kRowBytes / 16;            // words of a key per lane
    static constexpr int kVW = kRowBytes / 32;            // words of a value per lane
    static constexpr int kMt = D / 16;                    // 16-channel tiles of O^T
    static constexpr int kGr = BITS == 8 && D == 128 ? 1 : 2;   // 16-token granules per group (registers bound it)
    static constexpr int kRows = 8 * NT;
    static constexpr int kStride = D + 4;                 // floats of a row in the merge buffer
    static constexpr int kSmem = kWarps * kRows * kStride * 4;
    static constexpr float kOff = BITS == 4 ? 8.0f : 128.0f;
};

struct Run {            // a run of items in one (sequence, row tile, head)
    int b, n, row0, hk, chunk0, chunks;
};

template <int D, int BITS, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) attn_rows_kernel(const RowsArgs p)
{
    using C = RowsCfg<D, BITS, NT>;
    extern __shared__ __align__(16) float merge[];       // [kWarps][rows][kStride]
    __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
    __shared__ long long s_scan[kWarps];
    __shared__ long long s_skip;
    __shared__ int s_b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const AttnBatch &a = p.a;
    const int capacity = a.table_pages * a.page_size;

    // items of sequence b; n and chunks are set
    auto items_of = [&](int b, int &n, int &chunks) -> long long {
        const int t0 = __ldg(a.cu + b), t1 = __ldg(a.cu + b + 1);
        n = t0 >= 0 && t1 <= p.T ? max(0, t1 - t0) : 0;
        if ((long long)n * p.G > p.few) n = 0;
        const int len = max(1, min(__ldg(a.kv_len + b), capacity));
        chunks = (len + kItem - 1) / kItem;
        return (long long)((n * p.G + C::kRows - 1) / C::kRows) * p.Hkv * chunks;
    };

    // ---- this CTA's items ----
    long long at, end;
    Run run;
    {
        const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
        long long mine = 0;
        int n, chunks;
        for (int b = b0; b < b1; ++b) mine += items_of(b, n, chunks);
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_scan[warp] = x;
        __syncthreads();
        long long before = x - mine, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        // no more CTAs than items: every CTA between a run's first and last one has a part of it
        const long long ctas = min((long long)gridDim.x, total);
        at = blockIdx.x < ctas ? total * blockIdx.x / ctas : 0;
        end = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : 0;
        if (at < end && at >= before && at < before + mine) {
            int b = b0;
            for (; b < b1; ++b) {
                const long long k = items_of(b, n, chunks);
                if (at < before + k) break;
                before += k;
            }
            s_b = b;
            s_skip = at - before;
        }
        if (threadIdx.x == 0) p.joined[blockIdx.x] = make_int4(-1, 0, 0, 0);
        __syncthreads();
        grid_launch_dependents();
        if (at >= end) return;
        run.b = s_b;
        items_of(run.b, run.n, run.chunks);
        const long long skip = s_skip;
        run.chunk0 = (int)(skip % run.chunks);
        run.hk = (int)(skip / run.chunks % p.Hkv);
        run.row0 = (int)(skip / run.chunks / p.Hkv) * C::kRows;
        // total is needed below for the first CTA of a run
        s_scan[0] = total;    // every thread has read s_scan; the next read is after a barrier
    }
    bool head = true;         // the CTA's first run

    while (at < end) {
        const int b = run.b, hk = run.hk, rows = run.n * p.G - run.row0;
        const int take = (int)min((long long)(run.chunks - run.chunk0), end - at);
        const int len = min(__ldg(a.kv_len + b), capacity), first = __ldg(a.kv_len + b) - run.n;
        const int t_seq = __ldg(a.cu + b);
        // the warp's tokens: an equal, contiguous share
        const int tok0 = run.chunk0 * kItem + warp * take * (kItem / kWarps);
        const int tok1 = min(tok0 + take * (kItem / kWarps), len);

        // ---- q fragments, sums, limits of the lane's columns ----
        uint32_t qf[NT][D / 16][2];
        float sq[NT][2], m[NT][2], l[NT][2], W[NT][2], k[NT][2];
        int see[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = 8 * t + g;
            const uint16_t *src = nullptr;
            if (row < rows) {
                const int r = run.row0 + row;
                src = p.q + (int64_t)(t_seq + r / p.G) * p.ldq + (size_t)(hk * p.G + r % p.G) * D;
            }
            float s = 0.0f;
            if (BITS == 4) {
#pragma unroll
                for (int j = 0; j < C::kKW; ++j) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (src) x = to_code_order(__ldg(reinterpret_cast<const uint4 *>(src + (D / 4) * c + 8 * j)));
                    qf[t][2 * j][0] = x.x;
                    qf[t][2 * j][1] = x.y;
                    qf[t][2 * j + 1][0] = x.z;
                    qf[t][2 * j + 1][1] = x.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < C::kKW; ++j) {
                    uint2 x = make_uint2(0, 0);
                    if (src) x = __ldg(reinterpret_cast<const uint2 *>(src + 64 * (j / 4) + 16 * c + 4 * (j % 4)));
                    qf[t][j][0] = x.x;
                    qf[t][j][1] = x.y;
                }
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const __half2 h = *reinterpret_cast<const __half2 *>(&qf[t][j][u]);
                    s += __half2float(h.x) + __half2float(h.y);
                }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int col = 8 * t + 2 * c + u;
                sq[t][u] = __shfl_sync(0xffffffffu, s, (2 * c + u) * 4) * p.scale_log2;
                see[t][u] = col < rows ? first + (run.row0 + col) / p.G + 1 : 0;
                m[t][u] = -INFINITY;
                l[t][u] = W[t][u] = k[t][u] = 0.0f;
            }
        }
        int see_min = see[0][0];
#pragma unroll
        for (int t = 0; t < NT; ++t) see_min = min(see_min, min(see[t][0], see[t][1]));
        see_min = __reduce_min_sync(0xffffffffu, see_min);

        float o[NT][C::kMt][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[t][mt][r] = 0.0f;

        // ---- the tokens, kGr granules of 16 at a time ----
        uint32_t kw[C::kGr][2][C::kKW], vw[C::kGr][4][C::kVW], kp[C::kGr][2], vp[C::kGr][2];
        uint32_t base[C::kGr], base1[C::kGr];            // cache row of a granule's first token, or kNone: this group's, the next's
        auto locate = [&](int tok, uint32_t (&bs)[C::kGr]) {
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                const int pos = tok + 16 * i;
                const int page = pos < tok1 ? page_of(a, b, pos) : -1;
                bs[i] = page < 0 ? kNone : ((uint32_t)page * p.Hkv + hk) * a.page_size + (pos & (a.page_size - 1));
            }
        };
        auto load_k = [&](const uint32_t (&bs)[C::kGr]) {
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                if (bs[i] == kNone) continue;
                const uint8_t *src = p.c.k_codes + (size_t)(bs[i] + g) * C::kRowBytes + (C::kKW >= 4 ? 16 : 4 * C::kKW) * c;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    load_words<C::kKW < 4 ? C::kKW : 4>(src + 8 * h * C::kRowBytes, kw[i][h]);
                    if (C::kKW == 8) load_words<4>(src + 8 * h * C::kRowBytes + 64, kw[i][h] + (C::kKW == 8 ? 4 : 0));
                    kp[i][h] = __ldg(reinterpret_cast<const uint32_t *>(p.c.k_par) + bs[i] + g + 8 * h);
                }
            }
        };
        auto load_v = [&](const uint32_t (&bs)[C::kGr]) {
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                if (bs[i] == kNone) continue;
                const uint8_t *src = p.c.v_codes + (size_t)(bs[i] + 2 * c) * C::kRowBytes + 4 * C::kVW * g;
#pragma unroll
                for (int u = 0; u < 4; ++u) load_words<C::kVW>(src + ((u & 1) + 8 * (u >> 1)) * C::kRowBytes, vw[i][u]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    vp[i][h] = __ldg(reinterpret_cast<const uint32_t *>(p.c.v_par) + bs[i] + g + 8 * h);
            }
        };
        locate(tok0, base);
        load_k(base);
        load_v(base);
        locate(tok0 + 16 * C::kGr, base1);
        for (int tok = tok0; tok < tok1; tok += 16 * C::kGr) {
            // scores, in log2 units
            float sc[C::kGr][NT][4];
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[i][t][r] = 0.0f;
                if (base[i] == kNone) continue;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t a0, a1, a2, a3;
                    if (BITS == 4) {
                        const uint32_t x = kw[i][0][j / 2] >> (8 * (j & 1)), y = kw[i][1][j / 2] >> (8 * (j & 1));
                        a0 = pair_lo(x);
                        a1 = pair_lo(y);
                        a2 = pair_hi(x);
                        a3 = pair_hi(y);
                    } else {
                        const uint32_t x = kw[i][0][j % C::kKW], y = kw[i][1][j % C::kKW];
                        a0 = bytes_lo(x);
                        a1 = bytes_lo(y);
                        a2 = bytes_hi(x);
                        a3 = bytes_hi(y);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(sc[i][t], a0, a1, a2, a3, qf[t][j][0], qf[t][j][1]);
                }
            }
            float top[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                float ks[2], km[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float s = half_bits_to_float((uint16_t)(kp[i][h] & 0xFFFFu));
                    km[h] = fmaf(C::kOff, s, half_bits_to_float((uint16_t)(kp[i][h] >> 16)));
                    ks[h] = s * p.scale_log2;
                }
                const bool edge = base[i] == kNone || tok + 16 * i + 16 > see_min;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float x = fmaf(sc[i][t][r], ks[r >> 1], km[r >> 1] * sq[t][r & 1]);
                        if (edge && (base[i] == kNone || tok + 16 * i + g + 8 * (r >> 1) >= see[t][r & 1])) x = -INFINITY;
                        sc[i][t][r] = x;
                        top[t][r & 1] = fmaxf(top[t][r & 1], x);
                    }
            }
            // the key registers are free: the next group's
            load_k(base1);
            bool grow = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) grow |= top[t][u] > m[t][u] + 8.0f;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float x = top[t][u];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float m1 = fmaxf(m[t][u], x);
                        const float keep = m[t][u] == -INFINITY ? 0.0f : exp2_fast(m[t][u] - m1);
                        m[t][u] = m1;
                        l[t][u] *= keep;
                        W[t][u] *= keep;
#pragma unroll
                        for (int mt = 0; mt < C::kMt; ++mt) {
                            o[t][mt][u] *= keep;
                            o[t][mt][2 + u] *= keep;
                        }
                    }
            }
            // weights: sc becomes p s k, top its maximum
#pragma unroll
            for (int t = 0; t < NT; ++t) top[t][0] = top[t][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                float vs[2], vm[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    vs[h] = half_bits_to_float((uint16_t)(vp[i][h] & 0xFFFFu));
                    vm[h] = fmaf(C::kOff, vs[h], half_bits_to_float((uint16_t)(vp[i][h] >> 16)));
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float x = sc[i][t][r];
                        const float w = x == -INFINITY ? 0.0f : exp2_fast(x - m[t][r & 1]);
                        l[t][r & 1] += w;
                        // (an unseen token's parameters may be anything)
                        W[t][r & 1] = w > 0.0f ? fmaf(w, vm[r >> 1], W[t][r & 1]) : W[t][r & 1];
                        sc[i][t][r] = w > 0.0f ? w * vs[r >> 1] : 0.0f;
                        top[t][r & 1] = fmaxf(top[t][r & 1], sc[i][t][r]);
                    }
            }
            bool over = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) over |= k[t][u] == 0.0f ? top[t][u] > 0.0f : top[t][u] * k[t][u] > 16384.0f;
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float x = top[t][u];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        // 2^-e for x in [2^e, 2^(e+1)), e held within 2^-100 .. 2^100; only ever downwards
                        const int e = min(max((int)(__float_as_uint(x) >> 23) - 127, -100), 100);
                        const float k1 = __uint_as_float((uint32_t)(127 - e) << 23);
                        const bool set = x > 0.0f && (k[t][u] == 0.0f || k1 < k[t][u]);
                        const float f = set && k[t][u] > 0.0f ? k1 / k[t][u] : 1.0f;
                        if (set) k[t][u] = k1;
#pragma unroll
                        for (int mt = 0; mt < C::kMt; ++mt) {
                            o[t][mt][u] *= f;
                            o[t][mt][2 + u] *= f;
                        }
                    }
            }
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                if (base[i] == kNone) continue;
                uint32_t pb[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const __half2 x = __floats2half2_rn(sc[i][t][2 * h] * k[t][0], sc[i][t][2 * h + 1] * k[t][1]);
                        pb[t][h] = transpose8x8(*reinterpret_cast<const uint32_t *>(&x));
                    }
                auto tile = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(o[t][mt], a0, a1, a2, a3, pb[t][0], pb[t][1]);
                };
#pragma unroll
                for (int w = 0; w < C::kVW; ++w) {
                    if (BITS == 4) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // bytes 2h, 2h + 1 of one token under those of the next
                            const uint32_t x = __byte_perm(vw[i][0][w], vw[i][1][w], h ? 0x7632 : 0x5410);
                            const uint32_t y = __byte_perm(vw[i][2][w], vw[i][3][w], h ? 0x7632 : 0x5410);
                            tile(4 * w + 2 * h, pair_lo(x), pair_hi(x), pair_lo(y), pair_hi(y));
                            tile(4 * w + 2 * h + 1, pair_lo(x >> 8), pair_hi(x >> 8), pair_lo(y >> 8), pair_hi(y >> 8));
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = __byte_perm(vw[i][0][w], vw[i][1][w], h ? 0x7362 : 0x5140);
                            const uint32_t y = __byte_perm(vw[i][2][w], vw[i][3][w], h ? 0x7362 : 0x5140);
                            tile(2 * w + h, bytes_lo(x), bytes_hi(x), bytes_lo(y), bytes_hi(y));
                        }
                    }
                }
            }
            load_v(base1);
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) base[i] = base1[i];
            locate(tok + 32 * C::kGr, base1);
        }

        // ---- merge the warps ----
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x = l[t][u], y = W[t][u];
#pragma unroll
                for (int sft = 4; sft < 32; sft <<= 1) {
                    x += __shfl_xor_sync(0xffffffffu, x, sft);
                    y += __shfl_xor_sync(0xffffffffu, y, sft);
                }
                l[t][u] = x;
                W[t][u] = y;
                if (g == 0) {
                    s_m[warp][8 * t + 2 * c + u] = m[t][u];
                    s_l[warp][8 * t + 2 * c + u] = x;
                }
            }
        __syncthreads();
        const long long total = s_scan[0];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int col = 8 * t + 2 * c + u;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][col]);
                const float f = m[t][u] == -INFINITY ? 0.0f : exp2_fast(m[t][u] - M);
                const float fk = k[t][u] > 0.0f ? f / k[t][u] : 0.0f, fw = f * W[t][u];
                float *dst = merge + (warp * C::kRows + col) * C::kStride;
#pragma unroll
                for (int mt = 0; mt < C::kMt; ++mt)
                    *reinterpret_cast<float2 *>(dst + 16 * mt + 2 * g) =
                        make_float2(fmaf(o[t][mt][u], fk, fw), fmaf(o[t][mt][2 + u], fk, fw));
            }
        __syncthreads();
        const bool whole = run.chunk0 == 0 && take == run.chunks;
        // a run that began in an earlier CTA is the CTA's first part, one that goes on in a later one its last
        float *part = p.part + ((size_t)blockIdx.x * 2 + (run.chunk0 > 0 ? 0 : 1)) * C::kRows * (D + 2);
        for (int e = threadIdx.x; e < C::kRows * (D / 2); e += kThreads) {
            const int col = e / (D / 2), x = e % (D / 2);             // the pair at 16 mt + 2 g: x = 8 mt + g
            if (col >= rows) continue;
            float M = -INFINITY, L = 0.0f, s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][col]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 y = *reinterpret_cast<const float2 *>(merge + (w * C::kRows + col) * C::kStride + 2 * x);
                s0 += y.x;
                s1 += y.y;
                L += s_m[w][col] == -INFINITY ? 0.0f : s_l[w][col] * exp2_fast(s_m[w][col] - M);
            }
            const int ch = (D / 8) * (x % 8) + 2 * (x / 8);
            if (whole) {
                const int r = run.row0 + col;
                const float inv = L > 0.0f ? 1.0f / L : 0.0f;
                const __half2 h = __floats2half2_rn(s0 * inv, s1 * inv);
                *reinterpret_cast<__half2 *>(p.out + (int64_t)(t_seq + r / p.G) * p.ldo + (size_t)(hk * p.G + r % p.G) * D + ch) = h;
            } else {
                *reinterpret_cast<float2 *>(part + col * (D + 2) + ch) = make_float2(s0, s1);
                if (x == 0) *reinterpret_cast<float2 *>(part + col * (D + 2) + D) = make_float2(M, L);
            }
        }
        if (threadIdx.x == 0 && head && run.chunk0 > 0 && run.chunk0 + take == run.chunks) {
            // the run that ends here began at item at - chunk0
            const long long i0 = at - run.chunk0;
            p.joined[blockIdx.x] = make_int4(b, run.row0, hk, (int)(((i0 + 1) * min((long long)gridDim.x, total) - 1) / total));
        }
        __syncthreads();
        // ---- the next run ----
        head = false;
        at += take;
        if (at < end) {
            run.chunk0 = 0;
            if (++run.hk == p.Hkv) {
                run.hk = 0;
                run.row0 += C::kRows;
                if (run.row0 >= run.n * p.G) {
                    run.row0 = 0;
                    do {
                        ++run.b;
                    } while (items_of(run.b, run.n, run.chunks) == 0);
                }
            }
        }
    }
}

// One CTA per CTA of the first kernel: joins the run that ended in its first
// part.  A thread takes channels, the parts in order.
template <int D, int NT>
__global__ void __launch_bounds__(D) attn_rows_join_kernel(const RowsArgs p)
{
    constexpr int kRows = 8 * NT;
    grid_dependency_wait();
    const int4 j = p.joined[blockIdx.x];
    if (j.x < 0) return;
    const int t_seq = __ldg(p.a.cu + j.x), n = __ldg(p.a.cu + j.x + 1) - t_seq, rows = min(kRows, n * p.G - j.y);
    const int ch = threadIdx.x;
    for (int col = blockIdx.y; col < rows; col += gridDim.y) {
        auto part = [&](int cta) {
            return p.part + (((size_t)cta * 2 + (cta == j.w ? 1 : 0)) * kRows + col) * (D + 2);
        };
        float M = -INFINITY, L = 0.0f, s = 0.0f;
        for (int cta = j.w; cta <= (int)blockIdx.x; ++cta) {
            const float *x = part(cta);
            const float m = x[D], l = x[D + 1], v = x[ch];
            if (m == -INFINITY) continue;
            const float m1 = fmaxf(M, m), f0 = M == -INFINITY ? 0.0f : exp2_fast(M - m1), f1 = exp2_fast(m - m1);
            M = m1;
            L = fmaf(L, f0, l * f1);
            s = fmaf(s, f0, v * f1);
        }
        const int r = j.y + col;
        p.out[(int64_t)(t_seq + r / p.G) * p.ldo + (size_t)(j.z * p.G + r % p.G) * D + ch] =
            float_to_half_bits(L > 0.0f ? s / L : 0.0f);
    }
}

int sm_count()
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

constexpr int kMaxCtas = 2 * 160;       // sizes the workspace: two CTAs per SM

template <int D, int BITS, int NT>
cudaError_t launch_rows(RowsArgs p, cudaStream_t stream)
{
    using C = RowsCfg<D, BITS, NT>;
    auto kernel = attn_rows_kernel<D, BITS, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = min(sm_count() * (NT == 1 ? 2 : 1), kMaxCtas);
    kernel<<<ctas, kThreads, C::kSmem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 4);
    cfg.blockDim = dim3(D);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_rows_join_kernel<D, NT>, p);
}

}  // namespace

size_t rows_workspace(int d)
{
    return (size_t)kMaxCtas * (sizeof(int4) + 2 * 16 * (d + 2) * sizeof(float));
}

cudaError_t launch_paged_rows(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                              const AttnBatch &a, int few, bool eight, float scale, uint16_t *out, int64_t ldo,
                              void *workspace, cudaStream_t stream)
{
    int4 *joined = reinterpret_cast<int4 *>(workspace);
    RowsArgs p{q, ldq, ldo, out, c, a, T, Hq, Hkv, Hq / Hkv, few, scale * 1.4426950408889634f,
               reinterpret_cast<float *>(joined + kMaxCtas), joined};
    if (d == 128) {
        if (c.bits == 4) return eight ? launch_rows<128, 4, 1>(p, stream) : launch_rows<128, 4, 2>(p, stream);
        return eight ? launch_rows<128, 8, 1>(p, stream) : launch_rows<128, 8, 2>(p, stream);
    }
    if (c.bits == 4) return eight ? launch_rows<64, 4, 1>(p, stream) : launch_rows<64, 4, 2>(p, stream);
    return eight ? launch_rows<64, 8, 1>(p, stream) : launch_rows<64, 8, 2>(p, stream);
}

}  // namespace qoq
