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
// A warp works alone on its own tokens, without block barriers, in
// warp-level MMAs (m16n8k16, FP32 sums; the rows as the 8-wide N dimension):
//     S^T[token][row]   = codes of K (A, tokens x channels) x q (B)
//     O^T[channel][row] = codes of V^T (A, channels x tokens) x p s (B)
// Which channel sits at which fragment position does not matter as long as
// q, and O's write-out, agree; so a lane reads neighbouring bytes of a key or
// a value.  The weights go from the layout of S^T to that of B by one 8x8
// transposition (movmatrix) each.  A ring of three stages of 32 tokens (16 for
// 8-bit heads of 128) per warp is filled by bulk copies, one per granule of 16
// tokens and array, each issued by the lane that looked the page up.
//
// Running maximum m, sum l and sum of p m' in FP32; m may lag behind by 2^8,
// so O is rescaled rarely.  The weights p s are rounded to FP16 (half a step
// each) after a power of two k, which follows the largest s, so that small
// scales do not underflow.
//
// Work: a run is a (sequence, row tile, KV head) with its tokens in granules
// of 16, in that order; each run also counts kSwitch granules for what it
// costs to begin and end one.  Warp w of P takes an equal, contiguous share
// of that line, so all warps do the same work whatever the lengths, and
// neither a barrier nor shared memory ties them.  A run within one warp's
// share is finished there; one that spans warps leaves a partial result in
// each, and a second kernel joins them, in order.  (An earlier form shared
// each run among the eight warps of a CTA and merged them in shared memory:
// 122 against XXX us for 64 sequences of 300 to 8191 tokens, because CTAs
// with short runs spent their time switching.)
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
constexpr int kSwitch = 2;              // granules that a run counts for its beginning and end
constexpr int kLeast = 4;               // granules of a warp's share, at least (a partial result costs about as much)
constexpr uint64_t kBudgetNs = 2000000000ull;

__device__ int g_rows_error;            // non-zero after a bounded wait ran out

struct RowsArgs {
    const uint16_t *q;
    int64_t ldq, ldo;
    uint16_t *out;
    AttnCache c;
    AttnBatch a;
    int T, Hq, Hkv, G;
    int few;            // sequences with more rows are another kernel's
    float scale_log2;   // scale * log2(e)
    uint32_t e6, e5;    // 0x64006400, 0x54005400: see pair_lo
    float *part;        // [P][2][rows][D + 4]: sums, maximum, sum of weights
    int4 *joined;       // [P]: (sequence or -1, first row, KV head, first warp) of the run that ends in warp w's share
                        // and began in an earlier one's
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

// (code - off) pairs of a word: 4 bits: nibbles (0, 4) and (1, 5) of the 16-bit halves' low bytes.  The exponent
// patterns e6 = 0x64006400 and e5 = 0x54005400 come in registers whose values the compiler does not know: a logic
// instruction has room for one constant, and with two it becomes two (a quarter of this kernel's instructions).
__device__ __forceinline__ uint32_t pair_lo(uint32_t x, uint32_t e6)
{
    return sub_h2((x & 0x000F000Fu) | e6, 0x64086408u);   // 1024 + c - 1032
}

__device__ __forceinline__ uint32_t pair_hi(uint32_t x, uint32_t e5)
{
    return sub_h2((x & 0x00F000F0u) | e5, 0x54805480u);   // 64 + c - 72
}

// 8 bits: bytes (0, 1) or (2, 3) of x
__device__ __forceinline__ uint32_t bytes_lo(uint32_t x, uint32_t e6)
{
    return sub_h2(__byte_perm(x, e6, 0x5150), 0x64806480u);
}

__device__ __forceinline__ uint32_t bytes_hi(uint32_t x, uint32_t e6)
{
    return sub_h2(__byte_perm(x, e6, 0x5352), 0x64806480u);
}

template <int N>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t *w)
{
    if (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x;
        w[1] = x.y;
    } else {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
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
    static constexpr int kGr = BITS == 8 && D == 128 ? 1 : 2;   // 16-token granules per stage
    static constexpr int kGroup = 16 * kGr;               // tokens
    static constexpr int kGranule = 16 * (2 * kRowBytes + 8);   // bytes: keys, values, their parameters
    static constexpr int kStage = kGr * kGranule;
    static constexpr int kStages = 3;
    static constexpr int kSmem = kWarps * kStages * kStage;     // 102 KB (d = 128): two CTAs per SM
    static constexpr int kRows = 8 * NT;
    static constexpr int kStride = D + 4;                 // floats of a partial row
    static constexpr float kOff = BITS == 4 ? 8.0f : 128.0f;
};

struct Run {
    int b, n, row0, hk, grains;
};

template <int D, int BITS, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) attn_rows_kernel(const RowsArgs p)
{
    using C = RowsCfg<D, BITS, NT>;
    extern __shared__ __align__(128) uint8_t smem[];    // [kWarps][kStages][kStage]
    __shared__ uint64_t s_bar[kWarps][C::kStages];
    __shared__ int abort_flag;
    __shared__ long long s_sum[kWarps], s_before[kThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const AttnBatch &a = p.a;
    const int capacity = a.table_pages * a.page_size;
    const uint32_t e6 = p.e6, e5 = p.e5;
    // neighbouring warps of the line sit on different SMs, so that a short line uses all of them
    const int me = warp * gridDim.x + blockIdx.x;

    // the line's length over sequence b; n and grains are set
    auto length_of = [&](int b, int &n, int &grains) -> long long {
        const int t0 = __ldg(a.cu + b), t1 = __ldg(a.cu + b + 1);
        n = t0 >= 0 && t1 <= p.T ? max(0, t1 - t0) : 0;
        if ((long long)n * p.G > p.few) n = 0;
        grains = (max(1, min(__ldg(a.kv_len + b), capacity)) + 15) / 16;
        return (long long)((n * p.G + C::kRows - 1) / C::kRows) * p.Hkv * (grains + kSwitch);
    };

    // ---- this warp's share ----
    long long at, end, total, ctas;
    Run run;
    {
        const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += length_of(b, run.n, run.grains);
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_sum[warp] = x;
        __syncthreads();
        total = 0;
        x -= mine;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) x += s_sum[w];
            total += s_sum[w];
        }
        s_before[threadIdx.x] = x;
        if (lane == 0) {
            p.joined[me] = make_int4(-1, 0, 0, 0);
            for (int i = 0; i < C::kStages; ++i) mbar_init(smem_addr(&s_bar[warp][i]), 1);
            fence_mbar_init();
        }
        if (threadIdx.x == 0) abort_flag = 0;
        __syncthreads();
        grid_launch_dependents();
        ctas = min((long long)gridDim.x * kWarps, (total + kLeast - 1) / kLeast);
        if (me >= ctas) return;
        at = total * me / ctas;
        end = total * (me + 1) / ctas;
        int lo = 0, hi = kThreads - 1;               // the last thread whose sequences begin at or before `at`
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_before[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        long long skip = at - s_before[lo];
        for (run.b = lo * per;; ++run.b) {
            const long long len = length_of(run.b, run.n, run.grains);
            if (skip < len) break;
            skip -= len;
        }
        const int unit = run.grains + kSwitch;
        const int r = (int)(skip / unit);
        run.hk = r % p.Hkv;
        run.row0 = r / p.Hkv * C::kRows;
        at -= skip % unit;                           // where the run begins; the share begins within it
    }
    long long from = total * me / ctas;              // where the warp's part of the run begins
    uint8_t *ring_ptr = smem + warp * C::kStages * C::kStage;
    const uint32_t ring = smem_addr(ring_ptr), bar = smem_addr(&s_bar[warp][0]);
    uint32_t staged = 0, used = 0;                   // stages issued and consumed by the warp so far
    uint32_t there = 0;                              // four bits per slot: which of its granules have a page
    bool failed = false;
    // byte selectors of the value pass
    const uint32_t pick[2] = {BITS == 4 ? (c & 1 ? 0x1054u : 0x5410u) : (c & 1 ? 0x1504u : 0x5140u),
                              BITS == 4 ? (c & 1 ? 0x3276u : 0x7632u) : (c & 1 ? 0x3726u : 0x7362u)};

    while (at < end) {
        const int b = run.b, hk = run.hk, rows = run.n * p.G - run.row0;
        // granules [g0, g1) of the run
        const int g0 = (int)max(0ll, from - at - kSwitch), g1 = (int)min((long long)run.grains, end - at - kSwitch);
        if (g0 < g1) {
        const int len = min(__ldg(a.kv_len + b), capacity), first = __ldg(a.kv_len + b) - run.n;
        const int t_seq = __ldg(a.cu + b);
        const int tok0 = 16 * g0, tok1 = min(16 * g1, len);

        // ---- q fragments, sums, limits of the lane's columns ----
        uint32_t qf[NT][D / 16][2];
        float sq[NT][2], m[NT][2], l[NT][2], W[NT][2];
        float k = 0.0f;                                  // power of two on the value scales; 0: none seen yet
        int see[NT][2], see_max = 0;
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
                see_max = max(see_max, see[t][u]);
                m[t][u] = -INFINITY;
                l[t][u] = W[t][u] = 0.0f;
            }
        }
        int see_min = see[0][0];
#pragma unroll
        for (int t = 0; t < NT; ++t) see_min = min(see_min, min(see[t][0], see[t][1]));
        see_min = __reduce_min_sync(0xffffffffu, see_min);
        see_max = __reduce_max_sync(0xffffffffu, see_max);

        float o[NT][C::kMt][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[t][mt][r] = 0.0f;

        // ---- the tokens, a stage of kGr granules of 16 at a time, kStages of them in flight ----
        // Copies of the n stages from `stage` on; lane (stage, granule, array) looks its page up and issues one.
        auto issue = [&](int stage, int n) {
            const int so = lane / (4 * C::kGr), gi = lane / 4 % C::kGr, kind = lane & 3;
            const int pos = tok0 + (stage + so) * C::kGroup + 16 * gi;
            const int page = so < n && pos < tok1 ? page_of(a, b, pos) : -1;
            const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
            const int slot = (int)((staged + so) % C::kStages);
            if (so < n && lane % (4 * C::kGr) == 0) {
                const uint32_t mine = have >> lane & (C::kGr == 1 ? 0x1u : 0x11u);
                if (mine) mbar_arrive_expect_tx(bar + 8 * slot, __popc(mine) * C::kGranule);
                else mbar_arrive(bar + 8 * slot);
            }
            __syncwarp();
            if (page >= 0) {
                const size_t row = ((size_t)page * p.Hkv + hk) * a.page_size + (pos & (a.page_size - 1));
                const bool val = kind & 1;
                const uint8_t *src = kind < 2 ? (val ? p.c.v_codes : p.c.k_codes) + row * C::kRowBytes
                                              : reinterpret_cast<const uint8_t *>(val ? p.c.v_par : p.c.k_par) + row * 4;
                const uint32_t dst = ring + slot * C::kStage +
                                     (kind < 2 ? (val * C::kGr + gi) * 16 * C::kRowBytes
                                               : 2 * C::kGr * 16 * C::kRowBytes + (val * C::kGr + gi) * 64);
                bulk_load(dst, src, kind < 2 ? 16 * C::kRowBytes : 64, bar + 8 * slot);
            }
#pragma unroll
            for (int i = 0; i < C::kStages; ++i)
                if (i < n) {
                    const int s = (int)((staged + i) % C::kStages);
                    there = (there & ~(0xFu << 4 * s)) | ((have >> 4 * C::kGr * i & 1u) | (have >> 4 * C::kGr * i >> 3 & 2u)) << 4 * s;
                }
            staged += n;
        };
        const int stages = (tok1 - tok0 + C::kGroup - 1) / C::kGroup;     // 0 for an empty context
        // (the last run's slots were read by ordinary loads and are refilled by asynchronous copies)
        fence_proxy_async_smem();
        __syncwarp();
        issue(0, min(stages, C::kStages));
        for (int stage = 0; stage < stages; ++stage, ++used) {
            const int tok = tok0 + stage * C::kGroup, slot = (int)(used % C::kStages);
            if (!__all_sync(0xffffffffu, wait_bounded(bar + 8 * slot, (uint32_t)(used / C::kStages) & 1, &abort_flag, kBudgetNs))) {
                failed = true;
                break;
            }
            const uint8_t *sk = ring_ptr + slot * C::kStage + g * C::kRowBytes + (C::kKW >= 4 ? 16 : 4 * C::kKW) * c;
            // (lanes of odd c read the second token of a pair first: fewer bank conflicts)
            const uint8_t *sv = ring_ptr + slot * C::kStage + (C::kGr * 16 + 2 * c + (c & 1)) * C::kRowBytes + 4 * C::kVW * g;
            const int flip = c & 1 ? -C::kRowBytes : C::kRowBytes;
            const uint32_t *sp = reinterpret_cast<const uint32_t *>(ring_ptr + slot * C::kStage + 2 * C::kGr * 16 * C::kRowBytes) + g;
            uint32_t kp[C::kGr][2], vp[C::kGr][2];
            bool gone[C::kGr];                               // the granule's page is absent
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                gone[i] = !(there >> (4 * slot + i) & 1u);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    kp[i][h] = sp[16 * i + 8 * h];
                    vp[i][h] = sp[16 * (C::kGr + i) + 8 * h];
                }
            }
            // scores, in log2 units
            float sc[C::kGr][NT][4];
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[i][t][r] = 0.0f;
                if (gone[i]) continue;
                uint32_t kw[2][C::kKW];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *src = sk + (16 * i + 8 * h) * C::kRowBytes;
                    lds_words<C::kKW < 4 ? C::kKW : 4>(src, kw[h]);
                    if (C::kKW == 8) lds_words<4>(src + 64, kw[h] + (C::kKW == 8 ? 4 : 0));
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t a0, a1, a2, a3;
                    if (BITS == 4) {
                        const uint32_t x = kw[0][j / 2] >> (8 * (j & 1)), y = kw[1][j / 2] >> (8 * (j & 1));
                        a0 = pair_lo(x, e6);
                        a1 = pair_lo(y, e6);
                        a2 = pair_hi(x, e5);
                        a3 = pair_hi(y, e5);
                    } else {
                        const uint32_t x = kw[0][j % C::kKW], y = kw[1][j % C::kKW];
                        a0 = bytes_lo(x, e6);
                        a1 = bytes_lo(y, e6);
                        a2 = bytes_hi(x, e6);
                        a3 = bytes_hi(y, e6);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(sc[i][t], a0, a1, a2, a3, qf[t][j][0], qf[t][j][1]);
                }
            }
            // Tokens that no row sees may hold anything: their parameters become zeros, so that nothing below is NaN.
            const bool edge = tok + C::kGroup > see_min || gone[0] || gone[C::kGr - 1];
            if (edge) {
#pragma unroll
                for (int i = 0; i < C::kGr; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (gone[i] || tok + 16 * i + g + 8 * h >= see_max) kp[i][h] = vp[i][h] = 0u;
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
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[i][t][r] = fmaf(sc[i][t][r], ks[r >> 1], km[r >> 1] * sq[t][r & 1]);
            }
            if (edge) {
#pragma unroll
                for (int i = 0; i < C::kGr; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (gone[i] || tok + 16 * i + g + 8 * (r >> 1) >= see[t][r & 1]) sc[i][t][r] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < C::kGr; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) top[t][r & 1] = fmaxf(top[t][r & 1], sc[i][t][r]);
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
            // value scales; k brings the largest seen into [2^5, 2^6), so that with p <= 2^8 the products fit FP16
            // and scales down to 2^-20 of the largest keep full precision
            float vs[C::kGr][2], vm[C::kGr][2], vmax = 0.0f;
#pragma unroll
            for (int i = 0; i < C::kGr; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    vs[i][h] = half_bits_to_float((uint16_t)(vp[i][h] & 0xFFFFu));
                    vm[i][h] = fmaf(C::kOff, vs[i][h], half_bits_to_float((uint16_t)(vp[i][h] >> 16)));
                    vmax = fmaxf(vmax, vs[i][h]);
                }
            if (__any_sync(0xffffffffu, k == 0.0f ? vmax > 0.0f : vmax * k >= 64.0f)) {
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 4));
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 8));
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 16));
                // vmax in [2^e, 2^(e+1)) (an FP16 number, normal in FP32): k = 2^(5-e)
                const float k1 = __uint_as_float((127u + 5u + 127u - (__float_as_uint(vmax) >> 23)) << 23);
                const float f = k1 / (k == 0.0f ? k1 : k);
                k = k1;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[t][mt][r] *= f;
            }
            // weights: sc becomes p s k
            float sub[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) sub[t][u] = m[t][u] == -INFINITY ? 0.0f : m[t][u];
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                const float vk[2] = {vs[i][0] * k, vs[i][1] * k};
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float w = exp2_fast(sc[i][t][r] - sub[t][r & 1]);
                        l[t][r & 1] += w;
                        W[t][r & 1] = fmaf(w, vm[i][r >> 1], W[t][r & 1]);
                        sc[i][t][r] = w * vk[r >> 1];
                    }
            }
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                if (gone[i]) continue;
                uint32_t pb[NT][2], vw[4][C::kVW];
#pragma unroll
                for (int u = 0; u < 4; ++u) lds_words<C::kVW>(sv + (16 * i + 8 * (u >> 1)) * C::kRowBytes + (u & 1 ? flip : 0), vw[u]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const __half2 x = __floats2half2_rn(sc[i][t][2 * h], sc[i][t][2 * h + 1]);
                        pb[t][h] = transpose8x8(*reinterpret_cast<const uint32_t *>(&x));
                    }
                auto tile = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(o[t][mt], a0, a1, a2, a3, pb[t][0], pb[t][1]);
                };
#pragma unroll
                for (int w = 0; w < C::kVW; ++w) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // 4 bits: bytes 2h, 2h + 1 of a token under those of the next; 8 bits: the two tokens' bytes in turn
                        const uint32_t x = __byte_perm(vw[0][w], vw[1][w], pick[h]), y = __byte_perm(vw[2][w], vw[3][w], pick[h]);
                        if (BITS == 4) {
                            tile(4 * w + 2 * h, pair_lo(x, e6), pair_hi(x, e5), pair_lo(y, e6), pair_hi(y, e5));
                            tile(4 * w + 2 * h + 1, pair_lo(x >> 8, e6), pair_hi(x >> 8, e5), pair_lo(y >> 8, e6), pair_hi(y >> 8, e5));
                        } else {
                            tile(2 * w + h, bytes_lo(x, e6), bytes_hi(x, e6), bytes_lo(y, e6), bytes_hi(y, e6));
                        }
                    }
                }
            }
            if (stage + C::kStages < stages) {
                fence_proxy_async_smem();
                __syncwarp();
                issue(stage + C::kStages, 1);
            }
        }
        if (failed) break;

        // ---- finish, or leave a partial result ----
        const bool begins = g0 == 0, ends = g1 == run.grains;
        // a part that began in an earlier warp's share is the warp's first (slot 0), one that goes on its last
        float *part = p.part + ((size_t)me * 2 + (begins ? 1 : 0)) * C::kRows * C::kStride;
        const float inv_k = k > 0.0f ? 1.0f / k : 0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x = l[t][u], y = W[t][u];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    x += __shfl_xor_sync(0xffffffffu, x, w);
                    y += __shfl_xor_sync(0xffffffffu, y, w);
                }
                const int col = 8 * t + 2 * c + u;
                if (col >= rows) continue;
                // the lane's channels: D / 8 * g + 2 mt, + 1
                float v[2 * C::kMt];
#pragma unroll
                for (int mt = 0; mt < C::kMt; ++mt) {
                    v[2 * mt] = fmaf(o[t][mt][u], inv_k, y);
                    v[2 * mt + 1] = fmaf(o[t][mt][2 + u], inv_k, y);
                }
                if (begins && ends) {
                    const float inv = x > 0.0f ? 1.0f / x : 0.0f;
                    const int r = run.row0 + col;
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + (int64_t)(t_seq + r / p.G) * p.ldo +
                                                           (size_t)(hk * p.G + r % p.G) * D + (D / 8) * g);
#pragma unroll
                    for (int i = 0; i < C::kMt / 4; ++i) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __half2 z = __floats2half2_rn(v[8 * i + 2 * e] * inv, v[8 * i + 2 * e + 1] * inv);
                            h[e] = *reinterpret_cast<const uint32_t *>(&z);
                        }
                        dst[i] = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else {
                    float *dst = part + col * C::kStride;
#pragma unroll
                    for (int i = 0; i < C::kMt / 2; ++i)
                        reinterpret_cast<float4 *>(dst + (D / 8) * g)[i] =
                            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (g == 0) *reinterpret_cast<float2 *>(dst + D) = make_float2(m[t][u], x);
                }
            }
        // the warp whose share holds the run's first granule
        if (lane == 0 && ends && !begins)
            p.joined[me] = make_int4(b, run.row0, hk, (int)(((at + kSwitch + 1) * ctas - 1) / total));
        }
        // ---- the next run ----
        at += run.grains + kSwitch;
        from = at;
        if (at < end) {
            if (++run.hk == p.Hkv) {
                run.hk = 0;
                run.row0 += C::kRows;
                if (run.row0 >= run.n * p.G) {
                    run.row0 = 0;
                    do {
                        ++run.b;
                    } while (length_of(run.b, run.n, run.grains) == 0);
                }
            }
        }
    }
    if (failed) {
        // a wait ran out: report it, and let the copies in flight land before the shared memory goes away
        if (lane == 0) atomicExch(&g_rows_error, 1);
        const uint64_t stop = global_timer_ns() + 200000000ull;
        for (; used < staged; ++used)
            while (!mbar_try_wait(bar + 8 * (used % C::kStages), (used / C::kStages) & 1) && global_timer_ns() < stop) {
            }
    }
}

// Joins the runs that span warps.  CTA (x, y) looks at eight warps' ends and
// takes rows 2y and 2y + 1 of each run that ended there; eight of its 16
// warps share a row's parts, four in flight at a time, and the sums are
// joined in order.  A lane holds D / 32 channels.
constexpr int kJoinThreads = 512;

template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) attn_rows_join_kernel(const RowsArgs p)
{
    constexpr int kRows = 8 * NT, kStride = D + 4, kN = D / 32;
    __shared__ float s_v[2][8][D];
    __shared__ float2 s_ml[2][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = warp >> 3, w8 = warp & 7;
    grid_dependency_wait();
    for (int e = 0; e < 8; ++e) {
        const int last = blockIdx.x * 8 + e;
        const int4 j = p.joined[last];
        if (j.x < 0) continue;
        const int t_seq = __ldg(p.a.cu + j.x), n = __ldg(p.a.cu + j.x + 1) - t_seq, rows = min(kRows, n * p.G - j.y);
        const int row = 2 * blockIdx.y + half;
        if (2 * (int)blockIdx.y >= rows) continue;           // the same for the whole CTA
        float v[kN], M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = 0.0f;
        if (row < rows) {
            for (int w = j.w + w8; w <= last; w += 32) {
                float y[4][kN];
                float2 ml[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    ml[u] = make_float2(-INFINITY, 0.0f);
                    if (w + 8 * u > last) continue;
                    const float *x = p.part + (((size_t)(w + 8 * u) * 2 + (w + 8 * u == j.w ? 1 : 0)) * kRows + row) * kStride;
                    ml[u] = *reinterpret_cast<const float2 *>(x + D);
#pragma unroll
                    for (int i = 0; i < kN; ++i) y[u][i] = x[32 * i + lane];
                }
                const float m1 = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
                if (m1 == -INFINITY) continue;
                const float f0 = M == -INFINITY ? 0.0f : exp2_fast(M - m1);
                M = m1;
                L *= f0;
#pragma unroll
                for (int i = 0; i < kN; ++i) v[i] *= f0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (ml[u].x == -INFINITY) continue;
                    const float f = exp2_fast(ml[u].x - m1);
                    L = fmaf(ml[u].y, f, L);
#pragma unroll
                    for (int i = 0; i < kN; ++i) v[i] = fmaf(y[u][i], f, v[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) s_v[half][w8][32 * i + lane] = v[i];
        if (lane == 0) s_ml[half][w8] = make_float2(M, L);
        __syncthreads();
        for (int x = threadIdx.x; x < 2 * D; x += kJoinThreads) {
            const int hf = x / D, ch = x % D, r = j.y + 2 * blockIdx.y + hf;
            if (2 * (int)blockIdx.y + hf >= rows) continue;
            float m = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) m = fmaxf(m, s_ml[hf][w].x);
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float f = s_ml[hf][w].x == -INFINITY ? 0.0f : exp2_fast(s_ml[hf][w].x - m);
                l = fmaf(s_ml[hf][w].y, f, l);
                o = fmaf(s_v[hf][w][ch], f, o);
            }
            p.out[(int64_t)(t_seq + r / p.G) * p.ldo + (size_t)(j.z * p.G + r % p.G) * D + ch] =
                float_to_half_bits(l > 0.0f ? o / l : 0.0f);
        }
        __syncthreads();
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
    const int ctas = min(sm_count() * (NT == 1 ? 2 : 1), NT == 1 ? kMaxCtas : kMaxCtas / 2);
    constexpr int smem = RowsCfg<D, BITS, NT>::kSmem;
    auto kernel = attn_rows_kernel<D, BITS, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<ctas, kThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the join's CTAs come up while the first kernel runs and wait for its end
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas * kWarps / 8, 4 * NT);
    cfg.blockDim = dim3(kJoinThreads);
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
    // 8 rows for each warp of two CTAs per SM, or 16 for each of one
    return (size_t)kMaxCtas * kWarps * (sizeof(int4) + 2 * 8 * (d + 4) * sizeof(float));
}

cudaError_t launch_paged_rows(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                              const AttnBatch &a, int few, bool eight, float scale, uint16_t *out, int64_t ldo,
                              void *workspace, cudaStream_t stream)
{
    int4 *joined = reinterpret_cast<int4 *>(workspace);
    RowsArgs p{q, ldq, ldo, out, c, a, T, Hq, Hkv, Hq / Hkv, few, scale * 1.4426950408889634f, 0x64006400u, 0x54005400u,
               reinterpret_cast<float *>(joined + kMaxCtas * kWarps), joined};
    if (d == 128) {
        if (c.bits == 4) return eight ? launch_rows<128, 4, 1>(p, stream) : launch_rows<128, 4, 2>(p, stream);
        return eight ? launch_rows<128, 8, 1>(p, stream) : launch_rows<128, 8, 2>(p, stream);
    }
    if (c.bits == 4) return eight ? launch_rows<64, 4, 1>(p, stream) : launch_rows<64, 4, 2>(p, stream);
    return eight ? launch_rows<64, 8, 1>(p, stream) : launch_rows<64, 8, 2>(p, stream);
}

cudaError_t read_and_clear_rows_error(int *value)
{
    *value = 0;
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rows_error, sizeof(int));
    if (e != cudaSuccess) return e;
    if (v) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_rows_error, &zero, sizeof(int));
    }
    *value = v;
    return e;
}

}  // namespace qoq
