// qoq_attn_rows.cu -- attention of few rows (a decode step: one new token,
// the query heads of a KV head) over the paged 4/8-bit cache.
//
// Bound: the cache's bytes, read once.  What has to stay below that is the
// instructions that turn codes into tensor-core operands, so a code is never
// scaled on its own: with x = s c + m per token,
//     score_j = s_j (q . c_j) + m_j sum(q)
//     out     = sum_j (p_j s_j) c'_j + sum_j p_j m'_j    (c' = c - off, m' = m + off s)
// the products run on the codes, and the scales touch one number per token.
// Values are centred (off: 8 or 128), because their sum's terms should cancel
// in the tensor core and not against sum p m'.
//
// A warp works alone on its own tokens, without block barriers, in
// warp-level MMAs with the rows as the 8-wide N dimension:
//     S^T[token][row]   = codes of K (A, tokens x channels) x q (B), m16n8k32 on
//                         integers, exact: the codes are 8-bit operands after one
//                         mask each (none for 8 bits; FP16 operands took four times
//                         the instructions), and q is three 8-bit digits, whole
//                         multiples of 2^-21 of the power of two below the row's
//                         largest |q|: nothing is lost of a channel down to 2^-11 of
//                         it, and of a smaller one less than FP32 sums lose.  (Two
//                         digits lose half of a small channel's bits as soon as one
//                         channel is 100 times the rest.)
//     O^T[channel][row] = codes of V^T (A, channels x tokens) x p s (B), m16n8k16, FP16
// Which channel sits at which fragment position does not matter as long as
// q, and O's write-out, agree; so a lane reads neighbouring bytes of a key or
// a value.  The weights go from the layout of S^T to that of B by one 8x8
// transposition (movmatrix) each.  Each warp has a ring of three stages of 32
// tokens (16 for 8-bit heads of 128), filled by asynchronous copies.
//
// Running maximum m, sum l and sum of p m' in FP32; m may lag behind by 2^8,
// so O is rescaled rarely.  The weights p s are rounded to FP16 (half a step
// each) after a power of two k, which follows the largest s, so that small
// scales do not underflow.
//
// Work: a run is a (sequence, row tile, KV head) with its tokens in granules
// of 16, in that order; each run also counts kSwitch granules for what it
// costs to begin and end one.  Warp w of P takes an equal, contiguous share
// of that line, so all warps do the same work whatever the lengths, and no
// barrier ties them.  A run within one warp's share is finished there; one
// that spans warps leaves a partial result in each.  The warps of a CTA that
// end up in the middle of one run join theirs in shared memory first, and a
// second kernel joins what is left, in order.  (An earlier form shared each
// run among the eight warps of a CTA: 122 us against 102 at that time for 64
// sequences of 300 to 8191 tokens, because CTAs with short runs spent their
// time switching.  Without the joining in the CTA: 88 against 78.)
//
// Measured: those 64 sequences (307 MB of cache, 8 heads of 128 in 4 bits)
// 85 us, 3.6 TB/s (80 with two digits of q); two of about 115,000 tokens in 8
// bits (457 MB) 96 us, 4.8 TB/s.  No pipe is full (issue slots 58%, ALU 50%,
// HBM 46% in the first): 16 warps of an SM do not hide the latencies of a
// granule's chain, from codes through scores and weights to values.
#include <cuda_fp16.h>

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
// The lowest digit's products sum to less than 2^22 (128 channels of 255 * 128): on top of the bits of 1.5 * 2^23 they
// are an FP32 number's last bits, and their conversion is a subtraction.
constexpr int kLowBase = 0x4B400000;
constexpr int kSwitch = 2;              // granules that a run counts for its beginning and end
constexpr int kLeast = 4;               // granules of a warp's share, at least (a partial result costs about as much)

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

// D (16 x 8, INT32) += A (16 x 32, UINT8, row) * B (32 x 8, INT8, col).
__device__ __forceinline__ void mma16832(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
    static constexpr int kStage = kGr * (32 * kRowBytes + 128); // bytes: keys, values, their parameters
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
    __shared__ long long s_sum[kWarps], s_before[kThreads], s_run[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const AttnBatch &a = p.a;
    const int capacity = a.table_pages * a.page_size;
    const uint32_t e6 = p.e6, e5 = p.e5;
    // the line's length over sequence b; n and grains are set
    auto length_of = [&](int b, int &n, int &grains) -> long long {
        const int t0 = __ldg(a.cu + b), t1 = __ldg(a.cu + b + 1);
        n = t0 >= 0 && t1 <= p.T ? max(0, t1 - t0) : 0;
        if ((long long)n * p.G > p.few) n = 0;
        grains = (max(1, min(__ldg(a.kv_len + b), capacity)) + 15) / 16;
        return (long long)((n * p.G + C::kRows - 1) / C::kRows) * p.Hkv * (grains + kSwitch);
    };

    // ---- this warp's share ----
    long long at = 0, end = 0, from = 0, total, ctas;
    int me;
    bool neighbours;
    Run run = {0, 0, 0, 0, 0};
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
        if (lane == 0) s_run[warp] = -1;
        __syncthreads();
        grid_launch_dependents();
        ctas = min((long long)gridDim.x * kWarps, (total + kLeast - 1) / kLeast);
        // the warps of a CTA are neighbours in the line; when it is short they are on different SMs
        neighbours = ctas == (long long)gridDim.x * kWarps;
        me = neighbours ? blockIdx.x * kWarps + warp : warp * gridDim.x + blockIdx.x;
        if (lane == 0) p.joined[me] = make_int4(-1, 0, 0, 0);
        if (me < ctas) {
        at = from = total * me / ctas;
        end = total * (me + 1) / ctas;
        int lo = 0, hi = kThreads - 1;               // the last thread whose sequences begin at or before `at`
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_before[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        long long skip = at - s_before[lo];
        for (run.b = lo * per; run.b < a.B; ++run.b) {
            const long long len = length_of(run.b, run.n, run.grains);
            if (skip < len) break;
            skip -= len;
        }
        const int unit = run.grains + kSwitch;
        const int r = (int)(skip / unit);
        run.hk = r % p.Hkv;
        run.row0 = r / p.Hkv * C::kRows;
        at -= skip % unit;                           // where the run begins; the share begins (`from`) within it
        if (run.b >= a.B) end = at;                  // (the sums ran over: rows counted in several sequences)
        }
    }
    uint8_t *ring_ptr = smem + warp * C::kStages * C::kStage;
    const uint32_t ring = smem_addr(ring_ptr);
    // the lane's parameter of a granule: token lane % 16, of the key or the value
    const int my_par = 2 * C::kGr * 16 * C::kRowBytes + (lane & 7) * 16 + ((lane >> 4) * 2 + (lane >> 3 & 1)) * 4;
    // byte selectors of the value pass
    const uint32_t pick[2] = {BITS == 4 ? (c & 1 ? 0x1054u : 0x5410u) : (c & 1 ? 0x1504u : 0x5140u),
                              BITS == 4 ? (c & 1 ? 0x3276u : 0x7632u) : (c & 1 ? 0x3726u : 0x7362u)};

    while (at < end) {
        const int b = run.b, hk = run.hk, rows = run.n * p.G - run.row0;
        // granules [g0, g1) of the run
        const int g0 = (int)max(0ll, from - at - kSwitch), g1 = (int)min((long long)run.grains, end - at - kSwitch);
        if (g0 < g1) {
        const int held = max(0, __ldg(a.kv_len + b)), len = min(held, capacity), first = held - run.n;
        const int t_seq = __ldg(a.cu + b);
        const int tok0 = 16 * g0, tok1 = min(16 * g1, len);

        // ---- q: three 8-bit digits per channel, sums, limits of the lane's columns ----
        uint32_t qf[NT][3][D / 32][2];                   // [.][digit, highest first][MMA step][fragment register]
        float sq[NT][2], qs[NT][2];                      // sum of q, value of a unit of its digits; log2 units
        float m[NT][2], l[NT][2], W[NT][2];
        float k = 0.0f;                                  // power of two on the value scales; 0: none seen yet
        int see[NT][2], see_min = 1 << 30, see_max = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = 8 * t + g;
            // the lane's channels in the order its key words expand to: byte i of step j's registers 0 and 1 are
            // 4 bits: (D/4) c + 8 j + 2 i and the next; 8 bits: byte i of words 2j and 2j + 1
            __half x[D / 32][2][4];
            {
                const uint16_t *src = nullptr;
                if (row < rows) {
                    const int r = run.row0 + row;
                    src = p.q + (int64_t)(t_seq + r / p.G) * p.ldq + (size_t)(hk * p.G + r % p.G) * D;
                }
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    uint4 y = make_uint4(0, 0, 0, 0);
                    if (src) {
                        const int ch = BITS == 4 ? (D / 4) * c + 8 * j : 64 * (j / 2) + 16 * c + 8 * (j % 2);
                        y = __ldg(reinterpret_cast<const uint4 *>(src + ch));
                    }
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const __half h = __ushort_as_half((uint16_t)(w[e / 2] >> (16 * (e & 1))));
                        if (BITS == 4) x[j][e & 1][e / 2] = h;
                        else x[j][e / 4][e & 3] = h;
                    }
                }
            }
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    top = max_nan(top, fabsf(__half2float(x[j][e / 4][e & 3])));
                }
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^e <= top (an FP16 number, normal in FP32; a row of zeros: as the smallest): in units of 2^(e - 21), or of
            // NaN where the row is not finite
            const bool finite = top <= 65504.0f;
            const int e = max((int)(__float_as_uint(top) >> 23), 127 - 24) - 127;
            const float inv = finite ? __uint_as_float((uint32_t)(127 + 21 - e) << 23) : 0.0f;
            const float unit = finite ? __uint_as_float((uint32_t)(127 - 21 + e) << 23) : __uint_as_float(0x7FC00000u);
            int s = 0;                                   // of the digits: q's rounding then meets s c + m, not s c alone
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t dig[3] = {0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int v = __float2int_rn(__half2float(x[j][h][i]) * inv);    // below 2^22 in size
                        const int v1 = (v + 128) >> 8, v2 = (v1 + 128) >> 8;             // v = 256 v1 + (-128 .. 127), and so on
                        s += v;
                        dig[0] |= (uint32_t)(v2 & 0xFF) << (8 * i);
                        dig[1] |= (uint32_t)(v1 & 0xFF) << (8 * i);
                        dig[2] |= (uint32_t)(v & 0xFF) << (8 * i);
                    }
#pragma unroll
                    for (int k = 0; k < 3; ++k) qf[t][k][j][h] = dig[k];
                }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int col = 8 * t + 2 * c + u;
                qs[t][u] = __shfl_sync(0xffffffffu, unit, (2 * c + u) * 4) * p.scale_log2;
                sq[t][u] = (float)__shfl_sync(0xffffffffu, s, (2 * c + u) * 4) * qs[t][u];
                const bool real = col < rows;            // others' results go nowhere
                see[t][u] = real ? first + (run.row0 + col) / p.G + 1 : 1 << 30;
                if (real) {
                    see_min = min(see_min, see[t][u]);
                    see_max = max(see_max, see[t][u]);
                }
                m[t][u] = -INFINITY;
                l[t][u] = W[t][u] = 0.0f;
            }
        }
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
        // Copies of one stage into slot `to`: every lane brings 16 bytes of each 512 of a granule's keys and values
        // and one parameter, to where the lane that needs a token's four finds them side by side.  Returns a bit per
        // granule that has a page.  (Bulk copies issued by single lanes take uniform registers: 80 instructions per
        // granule against 20.)
        auto copy = [&](int tok, int to) -> uint32_t {
            uint32_t have = 0;
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                const int pos = tok + 16 * i, page = pos < tok1 ? page_of(a, b, pos) : -1;
                if (page >= 0) {
                    have |= 1u << i;
                    const uint32_t row = ((uint32_t)page * p.Hkv + hk) * a.page_size + (pos & (a.page_size - 1));
                    const uint8_t *kc = p.c.k_codes + (size_t)row * C::kRowBytes + 16 * lane;
                    const uint8_t *vc = p.c.v_codes + (size_t)row * C::kRowBytes + 16 * lane;
                    const uint32_t dk = ring + to * C::kStage + i * 16 * C::kRowBytes + 16 * lane;
                    const uint32_t dv = dk + C::kGr * 16 * C::kRowBytes;
#pragma unroll
                    for (int e = 0; e < 16 * C::kRowBytes; e += 512) {
                        cp_async<16>(dk + e, kc + e);
                        cp_async<16>(dv + e, vc + e);
                    }
                    cp_async<4>(ring + to * C::kStage + my_par + 128 * i,
                                reinterpret_cast<const uint32_t *>(lane < 16 ? p.c.k_par : p.c.v_par) + row + (lane & 15));
                }
            }
            cp_async_commit();
            return have;
        };
        const int stages = (tok1 - tok0 + C::kGroup - 1) / C::kGroup;     // 0 for an empty context
        uint32_t there = 0;                              // four bits per stage, the next one lowest: its granules have a page
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) there |= copy(tok0 + i * C::kGroup, i) << (4 * i);
        int slot = 0;
        for (int stage = 0; stage < stages; ++stage) {
            const int tok = tok0 + stage * C::kGroup;
            // the slot that the last stage left is filled again
            there |= copy(tok + (C::kStages - 1) * C::kGroup, slot == 0 ? C::kStages - 1 : slot - 1) << (4 * (C::kStages - 1));
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint8_t *sk = ring_ptr + slot * C::kStage + g * C::kRowBytes + (C::kKW >= 4 ? 16 : 4 * C::kKW) * c;
            // (lanes of odd c read the second token of a pair first: fewer bank conflicts)
            const uint8_t *sv = ring_ptr + slot * C::kStage + (C::kGr * 16 + 2 * c + (c & 1)) * C::kRowBytes + 4 * C::kVW * g;
            const int flip = c & 1 ? -C::kRowBytes : C::kRowBytes;
            const uint4 *sp = reinterpret_cast<const uint4 *>(ring_ptr + slot * C::kStage + 2 * C::kGr * 16 * C::kRowBytes) + g;
            uint32_t kp[C::kGr][2], vp[C::kGr][2];
            bool gone[C::kGr];                               // the granule's page is absent
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                gone[i] = !(there >> i & 1u);
                const uint4 x = sp[8 * i];
                kp[i][0] = x.x;
                kp[i][1] = x.y;
                vp[i][0] = x.z;
                vp[i][1] = x.w;
            }
            // q . codes: each digit's products exact in 32-bit integers, and joined in FP32
            float dot[C::kGr][NT][4];
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                int acc[NT][3][4];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 12; ++r) acc[t][r / 4][r % 4] = r < 8 ? 0 : kLowBase;
                uint32_t kw[2][C::kKW];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *src = sk + (16 * i + 8 * h) * C::kRowBytes;
                    lds_words<C::kKW < 4 ? C::kKW : 4>(src, kw[h]);
                    if (C::kKW == 8) lds_words<4>(src + 64, kw[h] + (C::kKW == 8 ? 4 : 0));
                }
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    uint32_t f[4];
                    if (BITS == 4) {
                        f[0] = kw[0][j % C::kKW] & 0x0F0F0F0Fu;
                        f[1] = kw[1][j % C::kKW] & 0x0F0F0F0Fu;
                        f[2] = kw[0][j % C::kKW] >> 4 & 0x0F0F0F0Fu;
                        f[3] = kw[1][j % C::kKW] >> 4 & 0x0F0F0F0Fu;
                    } else {
                        f[0] = kw[0][2 * j % C::kKW];
                        f[1] = kw[1][2 * j % C::kKW];
                        f[2] = kw[0][(2 * j + 1) % C::kKW];
                        f[3] = kw[1][(2 * j + 1) % C::kKW];
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int k = 0; k < 3; ++k) mma16832(acc[t][k], f, qf[t][k][j][0], qf[t][k][j][1]);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        dot[i][t][r] = fmaf((float)(acc[t][0][r] * 256 + acc[t][1][r]), 256.0f,
                                            __int_as_float(acc[t][2][r]) - __int_as_float(kLowBase));
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
            // scores in log2 units, above the maximum in use
            float sc[C::kGr][NT][4], base[NT][2], top[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    base[t][u] = m[t][u] == -INFINITY ? 0.0f : -m[t][u];
                    top[t][u] = -INFINITY;
                }
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                float ks[2], km[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ks[h] = half_bits_to_float((uint16_t)(kp[i][h] & 0xFFFFu));
                    km[h] = half_bits_to_float((uint16_t)(kp[i][h] >> 16));
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        sc[i][t][r] = fmaf(dot[i][t][r], ks[r >> 1] * qs[t][r & 1], fmaf(km[r >> 1], sq[t][r & 1], base[t][r & 1]));
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
                for (int u = 0; u < 2; ++u) grow |= m[t][u] == -INFINITY ? top[t][u] > -INFINITY : top[t][u] > 8.0f;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float x = top[t][u];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        // by how much the maximum in use grows (from 0 while there is none)
                        const float up = m[t][u] == -INFINITY ? (x == -INFINITY ? 0.0f : x) : fmaxf(x, 0.0f);
                        const float keep = m[t][u] == -INFINITY ? 1.0f : exp2_fast(-up);
                        if (x > -INFINITY) m[t][u] = (m[t][u] == -INFINITY ? 0.0f : m[t][u]) + up;
                        l[t][u] *= keep;
                        W[t][u] *= keep;
#pragma unroll
                        for (int mt = 0; mt < C::kMt; ++mt) {
                            o[t][mt][u] *= keep;
                            o[t][mt][2 + u] *= keep;
                        }
#pragma unroll
                        for (int i = 0; i < C::kGr; ++i) {
                            sc[i][t][u] -= up;
                            sc[i][t][2 + u] -= up;
                        }
                    }
            }
            // Value scales; k brings the largest seen into [2^5, 2^6), so that with p <= 2^8 the products p s k fit FP16.
            // In units of the largest scale, p s has FP16's full precision from 2^-19 on and vanishes below 2^-30: of a
            // token's values only what sets them apart from its m', whose sum is FP32 (2^17 such tokens together move
            // the output by less than 2^-13 of the largest token's range).
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
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
                const float vk[2] = {vs[i][0] * k, vs[i][1] * k};
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float w = exp2_fast(sc[i][t][r]);
                        l[t][r & 1] += w;
                        W[t][r & 1] = fmaf(w, vm[i][r >> 1], W[t][r & 1]);
                        sc[i][t][r] = w * vk[r >> 1];
                    }
            }
#pragma unroll
            for (int i = 0; i < C::kGr; ++i) {
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
            there >>= 4;
            slot = slot + 1 == C::kStages ? 0 : slot + 1;
            __syncwarp();
        }
        cp_async_wait<0>();
        __syncwarp();

        // ---- finish, or leave a partial result ----
        const bool begins = g0 == 0, ends = g1 == run.grains;
        // a part that began in an earlier warp's share is the warp's first (slot 0), one that goes on its last
        float *part = p.part + ((size_t)me * 2 + (begins ? 1 : 0)) * C::kRows * C::kStride;
        // a share in the middle of a run: the CTA's warps in that position join their parts first (below)
        const bool middle = neighbours && !begins && !ends;
        if (middle) {
            part = reinterpret_cast<float *>(ring_ptr);
            if (lane == 0) s_run[warp] = at;
        }
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
                    const float inv = x == 0.0f ? 0.0f : 1.0f / x;      // (not for a sum that is NaN)
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
                    // (a sum that is NaN counts whatever its maximum: the joins skip parts that saw nothing by theirs)
                    if (g == 0) *reinterpret_cast<float2 *>(dst + D) = make_float2(x == x ? m[t][u] : 0.0f, x);
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
                    } while (run.b < a.B && length_of(run.b, run.n, run.grains) == 0);
                    if (run.b >= a.B) break;         // (the sums ran over: rows counted in several sequences)
                }
            }
        }
    }
    // ---- warps in the middle of one run: their parts become one, the others' are marked empty ----
    __syncthreads();
    const long long mine = s_run[warp];
    if (mine >= 0) {
        int w0 = warp, w1 = warp + 1;
        while (w0 > 0 && s_run[w0 - 1] == mine) --w0;
        while (w1 < kWarps && s_run[w1] == mine) ++w1;
        float *out = p.part + (size_t)me * 2 * C::kRows * C::kStride;
        float *first = out - (size_t)(warp - w0) * 2 * C::kRows * C::kStride;   // the first of these warps' part
        for (int r = warp - w0; r < C::kRows; r += w1 - w0) {
            float M = -INFINITY, L = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            auto row = [&](int w) { return reinterpret_cast<const float *>(smem + w * C::kStages * C::kStage) + r * C::kStride; };
            for (int w = w0; w < w1; ++w) M = fmaxf(M, row(w)[D]);
            for (int w = w0; w < w1; ++w) {
                const float m = row(w)[D], f = m == -INFINITY ? 0.0f : exp2_fast(m - M);
                L = fmaf(row(w)[D + 1], f, L);
                if (lane < D / 4) {
                    const float4 y = reinterpret_cast<const float4 *>(row(w))[lane];
                    v = make_float4(fmaf(y.x, f, v.x), fmaf(y.y, f, v.y), fmaf(y.z, f, v.z), fmaf(y.w, f, v.w));
                }
            }
            if (lane < D / 4) reinterpret_cast<float4 *>(first + r * C::kStride)[lane] = v;
            if (lane == 0) *reinterpret_cast<float2 *>(first + r * C::kStride + D) = make_float2(M, L);
        }
        if (warp > w0 && lane < C::kRows) *reinterpret_cast<float2 *>(out + lane * C::kStride + D) = make_float2(-INFINITY, 0.0f);
    }
}

// Joins the runs that span warps: CTA x the run that ended in warp x's share, one row per warp.  The lanes weigh 128
// parts at a time, the parts that are not empty go into a list, and the warp adds those, in order, eight loads at a time
// (a chain of loads is all that this kernel is), a lane holding four channels.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) attn_rows_join_kernel(const RowsArgs p)
{
    constexpr int kRows = 8 * NT, kStride = D + 4, kParts = 128, kAhead = 8;
    __shared__ int s_part[kWarps][kParts];
    __shared__ float s_f[kWarps][kParts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    const int last = blockIdx.x;
    const int4 j = p.joined[last];
    if (j.x < 0) return;
    const int t_seq = __ldg(p.a.cu + j.x), n = __ldg(p.a.cu + j.x + 1) - t_seq, rows = min(kRows, n * p.G - j.y);
    for (int row = warp; row < rows; row += kWarps) {
        const float *parts = p.part + row * kStride;
        auto part = [&](int w) { return parts + ((size_t)w * 2 + (w == j.w ? 1 : 0)) * kRows * kStride; };
        float M = -INFINITY, L = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w0 = j.w; w0 <= last; w0 += kParts) {
            float2 ml[kParts / 32];
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kParts / 32; ++k) {
                const int w = w0 + 32 * k + lane;
                ml[k] = w <= last ? *reinterpret_cast<const float2 *>(part(w) + D) : make_float2(-INFINITY, 0.0f);
            }
#pragma unroll
            for (int k = 0; k < kParts / 32; ++k) top = fmaxf(top, ml[k].x);
            const float m1 = fmaxf(M, warp_max(top));
            if (m1 == -INFINITY) continue;
            const float f0 = M == -INFINITY ? 0.0f : exp2_fast(M - m1);
            float l = 0.0f;
            int count = 0;
            __syncwarp();                                    // the list has been read
#pragma unroll
            for (int k = 0; k < kParts / 32; ++k) {
                const float f = ml[k].x == -INFINITY ? 0.0f : exp2_fast(ml[k].x - m1);
                l += ml[k].y * f;
                const uint32_t some = __ballot_sync(0xffffffffu, f > 0.0f);
                if (f > 0.0f) {
                    const int at = count + __popc(some & ((1u << lane) - 1));
                    s_part[warp][at] = w0 + 32 * k + lane;
                    s_f[warp][at] = f;
                }
                count += __popc(some);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            M = m1;
            L = fmaf(L, f0, l);
            v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
            __syncwarp();
            for (int i = 0; i < count; i += kAhead) {
                float4 y[kAhead];
                float g[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    g[u] = 0.0f;
                    y[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i + u < count) {
                        g[u] = s_f[warp][i + u];
                        if (lane < D / 4) y[u] = reinterpret_cast<const float4 *>(part(s_part[warp][i + u]))[lane];
                    }
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    v = make_float4(fmaf(y[u].x, g[u], v.x), fmaf(y[u].y, g[u], v.y), fmaf(y[u].z, g[u], v.z),
                                    fmaf(y[u].w, g[u], v.w));
            }
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const int r = j.y + row;
        const __half2 h0 = __floats2half2_rn(v.x * inv, v.y * inv), h1 = __floats2half2_rn(v.z * inv, v.w * inv);
        if (lane < D / 4)
            *reinterpret_cast<uint2 *>(p.out + (int64_t)(t_seq + r / p.G) * p.ldo + (size_t)(j.z * p.G + r % p.G) * D + 4 * lane) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
    }
}

constexpr int kMaxCtas = 2 * 160;       // sizes the workspace: two CTAs per SM

template <int D, int BITS, int NT>
cudaError_t launch_rows(const RowsArgs &p, cudaStream_t stream, bool join)
{
    const int ctas = min(attn_sms() * (NT == 1 ? 2 : 1), NT == 1 ? kMaxCtas : kMaxCtas / 2);
    // (the join's CTAs come up as the others end, and wait for the last)
    if (join) return launch_kernel(attn_rows_join_kernel<D, NT>, dim3(ctas * kWarps), kThreads, 0, stream, true, p);
    constexpr int smem = RowsCfg<D, BITS, NT>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<D, BITS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(attn_rows_kernel<D, BITS, NT>, dim3(ctas), kThreads, smem, stream, false, p);
}

}  // namespace

size_t rows_workspace(int d)
{
    // 8 rows for each warp of two CTAs per SM, or 16 for each of one
    return (size_t)kMaxCtas * kWarps * (sizeof(int4) + 2 * 8 * (d + 4) * sizeof(float));
}

cudaError_t launch_paged_rows(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                              const AttnBatch &a, int few, bool eight, float scale, uint16_t *out, int64_t ldo,
                              void *workspace, cudaStream_t stream, bool join)
{
    int4 *joined = reinterpret_cast<int4 *>(workspace);
    RowsArgs p{q, ldq, ldo, out, c, a, T, Hq, Hkv, Hq / Hkv, few, scale * 1.4426950408889634f, 0x64006400u, 0x54005400u,
               reinterpret_cast<float *>(joined + kMaxCtas * kWarps), joined};
    if (d == 128) {
        if (c.bits == 4) return eight ? launch_rows<128, 4, 1>(p, stream, join) : launch_rows<128, 4, 2>(p, stream, join);
        return eight ? launch_rows<128, 8, 1>(p, stream, join) : launch_rows<128, 8, 2>(p, stream, join);
    }
    if (c.bits == 4) return eight ? launch_rows<64, 4, 1>(p, stream, join) : launch_rows<64, 4, 2>(p, stream, join);
    return eight ? launch_rows<64, 8, 1>(p, stream, join) : launch_rows<64, 8, 2>(p, stream, join);
}

}  // namespace qoq
