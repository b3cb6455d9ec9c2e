// qoq_cache.cu -- rotary positions, the paged 4/8-bit key/value cache's
// writer (with the rotation fused in) and its reader.
//
// All three move rows of heads once, and HBM is their floor.  A "slot" is the
// unit of work: one thread, 16 channels of a head row in two 16-byte
// vectors chosen so that the thread holds both channels of its 8 rotation
// pairs: slot j takes pairs 8j .. 8j + 7, i.e. vectors j and j + rot/16
// (half layout) or 2j and 2j + 1 (interleaved, and the channels from rot
// on).  d / 16 neighbouring lanes make a head row, so the row's minimum and
// maximum for the quantiser are shuffles away.
//
// A rotation is the FP64 result rounded to FP16 once.  FP32 angles are off by
// up to pos * freq * 2^-24 (0.06 rad at position 2^20), so the angle's fraction
// of a turn is taken in FP64 (sincospi then needs no range reduction); and an
// FP32 rotation lands on the wrong side of an FP16 rounding boundary about
// once in 4000 values, which would make the fused writer's codes differ from
// a rotation followed by a write.  So it is computed in FP32 with a bound on
// its error, and again in FP64 only where the bound reaches a boundary: the
// same bits as FP64 throughout, without its four conversions per pair, which
// a quarter-rate pipe does (an append of 12000 tokens, 48 heads:
// 72 us against 154).
//
// None of the three fills the pipes or HBM: a thread has one slot's loads in
// flight (the append: issue slots 70%, HBM 37%, the first stall is that on
// loads).
//
// Likewise the quantiser multiplies by the reciprocal of the scale, and takes
// the IEEE division only next to a rounding boundary.
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "qoq_attn_device.cuh"
#include "qoq_attn_internal.h"
#include "qoq_quant.cuh"

namespace qoq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;          // tokens per CTA
constexpr int kMaxReadTok = 16;     // the same for the reader

// (amplitude * cos, amplitude * sin) of position pos at frequency f.
__device__ __forceinline__ double2 turn(int pos, double f, float amplitude)
{
    double t = (double)pos * (f * 0.15915494309189535);    // f / (2 pi): turns
    t -= rint(t);
    double s, c;
    sincospi(2.0 * t, &s, &c);
    return make_double2(amplitude * c, amplitude * s);
}

// The vector (8 channels) indices of slot j.
__device__ __forceinline__ int2 slot_vectors(int j, int rot, int interleaved)
{
    return j < rot / 16 && !interleaved ? make_int2(j, j + rot / 16) : make_int2(2 * j, 2 * j + 1);
}

__device__ __forceinline__ float2 halves(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

__device__ __forceinline__ uint32_t to_halves(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Cosines and sines of a token's rotation pairs, times the amplitude, in FP32 and (after them) FP64: pair 8 j + i, the
// i-th of slot j, is entry i * slots + j, so that neighbouring slots' lanes read neighbouring entries.
struct Turns {
    const float2 *fast;
    const double2 *exact;
    int slots;
};

// Two pairs (x1, x2) and (z1, z2), turned by entries is and it, as two FP16 words: (y1, w1), (y2, w2), or (y1, y2), (w1, w2) when
// INTER (y: the first pair turned, w: the second).  The FP32 results are off by at most 2^-24 (|x1 c| + 2 |x2 s| + |y|)
// (each factor's rounding, the product's, the sum's) < bound * max(|x1|, |x2|).
template <bool INTER>
__device__ __forceinline__ void turn2(float x1, float x2, float z1, float z2, const Turns &c, int is, int it, float bound,
                                      uint32_t &o0, uint32_t &o1)
{
    const float2 s = c.fast[is * c.slots], t = c.fast[it * c.slots];
    const float y1 = fmaf(x1, s.x, -(x2 * s.y)), y2 = fmaf(x1, s.y, x2 * s.x);
    const float w1 = fmaf(z1, t.x, -(z2 * t.y)), w2 = fmaf(z1, t.y, z2 * t.x);
    const float ey = bound * fmaxf(fabsf(x1), fabsf(x2)), ew = bound * fmaxf(fabsf(z1), fabsf(z2));
    uint32_t l0, l1;
    if (INTER) {
        l0 = to_halves(y1 - ey, y2 - ey);
        o0 = to_halves(y1 + ey, y2 + ey);
        l1 = to_halves(w1 - ew, w2 - ew);
        o1 = to_halves(w1 + ew, w2 + ew);
    } else {
        l0 = to_halves(y1 - ey, w1 - ew);
        o0 = to_halves(y1 + ey, w1 + ew);
        l1 = to_halves(y2 - ey, w2 - ew);
        o1 = to_halves(y2 + ey, w2 + ew);
    }
    if (l0 != o0 || l1 != o1) {
        const double2 d = c.exact[is * c.slots], f = c.exact[it * c.slots];
        const double a1 = x1, a2 = x2, b1 = z1, b2 = z2;
        const __half h1 = __double2half(fma(a1, d.x, -(a2 * d.y)));
        const __half h2 = __double2half(fma(a1, d.y, a2 * d.x));
        const __half g1 = __double2half(fma(b1, f.x, -(b2 * f.y)));
        const __half g2 = __double2half(fma(b1, f.y, b2 * f.x));
        const __half2 p = INTER ? __halves2half2(h1, h2) : __halves2half2(h1, g1);
        const __half2 q = INTER ? __halves2half2(g1, g2) : __halves2half2(h2, g2);
        o0 = *reinterpret_cast<const uint32_t *>(&p);
        o1 = *reinterpret_cast<const uint32_t *>(&q);
    }
}

// Rotates the 8 pairs of a slot (a, b: its two vectors); c points at the slot's first entries.
template <bool INTER>
__device__ __forceinline__ void rotate_slot(uint4 &a, uint4 &b, const Turns &c, float bound)
{
    uint32_t *u = &a.x, *v = &b.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = halves(u[i]), q = halves(v[i]);
        if (INTER) {
            // word i of a is pair i, word i of b pair 4 + i
            turn2<true>(p.x, p.y, q.x, q.y, c, i, 4 + i, bound, u[i], v[i]);
        } else {
            // words i hold channels 2i, 2i + 1 of either half
            turn2<false>(p.x, q.x, p.y, q.y, c, 2 * i, 2 * i + 1, bound, u[i], v[i]);
        }
    }
}

// Fills a token's tables, pairs first, first + step, ...
__device__ __forceinline__ void make_turns(float2 *fast, double2 *exact, int pos, const AttnRotary &r, int first, int step)
{
    for (int e = first; e < r.rot / 2; e += step) {
        const double2 t = turn(pos, __ldg(r.freq + e), r.amplitude);
        const int at = e % 8 * (r.rot / 16) + e / 8;
        exact[at] = t;
        fast[at] = make_float2((float)t.x, (float)t.y);
    }
}

// bound of turn2 for this amplitude: 2^-24 * (1 + 2 + sqrt 2) < 2^-21.8
__device__ __forceinline__ float turn_bound(float amplitude)
{
    return 4e-7f * fabsf(amplitude);
}

// ---------------------------------------------------------------- rotary --
template <bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const uint16_t *x, int64_t ldx,
                                                          const int32_t *__restrict__ pos, AttnRotary r, int T, int H,
                                                          int d, int tb, uint16_t *y, int64_t ldy)
{
    extern __shared__ __align__(16) double2 exact[];     // [tb][rot / 2], then fast the same
    const int t0 = blockIdx.x * tb, n = min(tb, T - t0), pairs = r.rot / 2;
    float2 *fast = reinterpret_cast<float2 *>(exact + tb * pairs);
    for (int i = threadIdx.x >> 6; i < n; i += kThreads >> 6)
        make_turns(fast + i * pairs, exact + i * pairs, __ldg(pos + t0 + i), r, threadIdx.x & 63, 64);
    __syncthreads();
    // A thread's slot stays the same, its head advances (without a division); threads past a multiple of the slots idle.
    const int slots = d / 16, rows = kThreads / slots, j = threadIdx.x % slots;
    if ((int)threadIdx.x >= rows * slots) return;
    const float bound = turn_bound(r.amplitude);
    const int2 at = slot_vectors(j, r.rot, INTER);
    for (int h = threadIdx.x / slots, i = 0;; h += rows) {
        while (h >= H) {
            h -= H;
            ++i;
        }
        if (i >= n) break;
        const uint4 *src = reinterpret_cast<const uint4 *>(x + (t0 + i) * ldx + (size_t)h * d);
        uint4 *dst = reinterpret_cast<uint4 *>(y + (t0 + i) * ldy + (size_t)h * d);
        uint4 va = src[at.x], vb = src[at.y];
        if (j < r.rot / 16)
            rotate_slot<INTER>(va, vb, {fast + i * pairs + j, exact + i * pairs + j, r.rot / 16}, bound);
        dst[at.x] = va;
        dst[at.y] = vb;
    }
}

// ---------------------------------------------------------------- append --
// Codes of the 8 channels of a vector as whole FP32 numbers: round((x - m) / s), at most 2^BITS - 1.  The product with
// the rounded reciprocal is off the IEEE quotient by less than 2^-21 of it, so the two round alike unless the product is
// within 2^-13 of a half.
template <int BITS>
__device__ __forceinline__ void codes8(const uint4 &v, float m, float s, float inv, float (&c)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = halves(w[i / 2]);
        const float q = ((i & 1 ? f.y : f.x) - m) * inv;
        c[i] = rintf(q);
        near |= fabsf(q - c[i]) > 0.5f - 0x1p-13f;
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = halves(w[i / 2]);
            c[i] = s == 0.0f ? 0.0f : rintf(__fdiv_rn((i & 1 ? f.y : f.x) - m, s));
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fminf(c[i], (float)((1 << BITS) - 1));
}

// Whole numbers below 256 to bytes: the low byte of x + 2^23.
__device__ __forceinline__ uint32_t bytes4(float a, float b, float c, float d)
{
    const uint32_t x = __float_as_uint(a + 8388608.0f), y = __float_as_uint(b + 8388608.0f);
    const uint32_t z = __float_as_uint(c + 8388608.0f), w = __float_as_uint(d + 8388608.0f);
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

template <int D, int BITS, bool INTER>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(
    const uint16_t *__restrict__ k, int64_t ldk, const uint16_t *__restrict__ v, int64_t ldv, const uint16_t *q,
    int64_t ldq, uint16_t *q_out, int64_t ldqo, int T, int Hq, int Hkv, AttnRotary r, AttnCache c, AttnBatch a, int tb)
{
    constexpr int kSlots = D / 16;
    __shared__ double2 exact[kMaxTok][D / 2];
    __shared__ float2 fast[kMaxTok][D / 2];
    __shared__ int s_pos[kMaxTok], s_page[kMaxTok];
    const int t0 = blockIdx.x * tb, n = min(tb, T - t0);
    if (threadIdx.x < n) {
        const int t = t0 + threadIdx.x, b = sequence_of(a.cu, a.B, t);
        const int pos = b < 0 ? 0 : __ldg(a.kv_len + b) - (__ldg(a.cu + b + 1) - t);
        s_pos[threadIdx.x] = pos;
        s_page[threadIdx.x] = b < 0 ? -2 : page_of(a, b, pos);   // -2: no sequence
    }
    __syncthreads();
    for (int i = threadIdx.x >> 6; i < n; i += kThreads >> 6)
        make_turns(fast[i], exact[i], s_pos[i], r, threadIdx.x & 63, 64);
    __syncthreads();
    const float bound = turn_bound(r.amplitude);
    const int H = Hq + 2 * Hkv;     // head rows of a token: q, then k, then v
    // A thread's slot stays the same, its head row advances (without a division).  Every lane takes part in the shuffles
    // of each pass; lanes past the end do nothing else.
    const int j = threadIdx.x % kSlots;
    int h = threadIdx.x / kSlots, i = 0;
    for (int e0 = 0; e0 < n * H * kSlots; e0 += kThreads, h += kThreads / kSlots) {
        while (h >= H) {
            h -= H;
            ++i;
        }
        const bool in = i < n;
        const int page = in ? s_page[i] : -2;
        const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hkv;
        const bool work = in && page != -2 && (is_q || page >= 0);
        const int rot = is_q || is_k ? r.rot : 0;
        const int2 at = slot_vectors(j, rot, INTER);
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (work) {
            const int t = t0 + i;
            const uint16_t *row = is_q ? q + t * ldq + (size_t)h * D
                                  : is_k ? k + t * ldk + (size_t)(h - Hq) * D
                                         : v + t * ldv + (size_t)(h - Hq - Hkv) * D;
            x = reinterpret_cast<const uint4 *>(row)[at.x];
            y = reinterpret_cast<const uint4 *>(row)[at.y];
            if (j < rot / 16) rotate_slot<INTER>(x, y, {fast[i] + j, exact[i] + j, r.rot / 16}, bound);
            if (is_q) {
                uint4 *dst = reinterpret_cast<uint4 *>(q_out + t * ldqo + (size_t)h * D);
                dst[at.x] = x;
                dst[at.y] = y;
            }
        }
        if (__all_sync(0xffffffffu, is_q || !work)) continue;
        // the row's minimum and maximum, as FP16 pairs
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        __half2 lo2 = *reinterpret_cast<const __half2 *>(&w[0]), hi2 = lo2;
#pragma unroll
        for (int u = 1; u < 8; ++u) {
            lo2 = __hmin2_nan(lo2, *reinterpret_cast<const __half2 *>(&w[u]));
            hi2 = __hmax2_nan(hi2, *reinterpret_cast<const __half2 *>(&w[u]));
        }
        float lo = min_nan(__low2float(lo2), __high2float(lo2)), hi = max_nan(__low2float(hi2), __high2float(hi2));
#pragma unroll
        for (int o = 1; o < kSlots; o <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (work && !is_q) {
            // A row that is not finite gets a scale and a minimum of NaN: all its values read back as that, and whoever
            // sees them knows.
            if (!(hi - lo <= 2 * 65504.0f)) lo = hi = __uint_as_float(0x7FC00000u);
            const __half sh = __float2half_rz(__fdiv_rn(hi - lo, (float)((1 << BITS) - 1)));
            const float s = __half2float(sh), inv = s == 0.0f ? 0.0f : __fdiv_rn(1.0f, s);
            const int hk = is_k ? h - Hq : h - Hq - Hkv;
            const size_t row = ((size_t)page * Hkv + hk) * a.page_size + (s_pos[i] & (a.page_size - 1));
            uint8_t *dst = (is_k ? c.k_codes : c.v_codes) + row * (D * BITS / 8);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float f[8];
                codes8<BITS>(u ? y : x, lo, s, inv, f);
                const int vec = u ? at.y : at.x;
                if (BITS == 4)
                    reinterpret_cast<uint32_t *>(dst)[vec] =
                        bytes4(fmaf(f[1], 16.0f, f[0]), fmaf(f[3], 16.0f, f[2]), fmaf(f[5], 16.0f, f[4]), fmaf(f[7], 16.0f, f[6]));
                else
                    reinterpret_cast<uint2 *>(dst)[vec] = make_uint2(bytes4(f[0], f[1], f[2], f[3]), bytes4(f[4], f[5], f[6], f[7]));
            }
            if (j == 0)
                reinterpret_cast<uint32_t *>(is_k ? c.k_par : c.v_par)[row] =
                    (uint32_t)__half_as_ushort(sh) | ((uint32_t)float_to_half_bits(lo) << 16);
        }
    }
}

// ------------------------------------------------------------------ read --
// A thread takes kAhead vectors of 8 channels at a time, all their loads before the first use.
template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(AttnCache c, AttnBatch a, int T, int Hkv, int tb,
                                                              uint32_t e6, uint32_t e4, uint16_t *__restrict__ K,
                                                              uint16_t *__restrict__ V)
{
    constexpr int kVecs = D / 8, kAhead = 4;
    __shared__ int s_off[kMaxReadTok], s_page[kMaxReadTok];
    const int t0 = blockIdx.x * tb, n = min(tb, T - t0);
    if (threadIdx.x < n) {
        const int t = t0 + threadIdx.x, b = sequence_of(a.cu, a.B, t);
        const int pos = b < 0 ? 0 : __ldg(a.kv_len + b) - (__ldg(a.cu + b + 1) - t);
        s_page[threadIdx.x] = b < 0 ? -2 : page_of(a, b, pos);
        s_off[threadIdx.x] = pos & (a.page_size - 1);
    }
    __syncthreads();
    // rows of a token: (head, key or value); a thread's vector stays the same, its row advances by constants
    const int rows = 2 * Hkv, j = threadIdx.x % kVecs;
    constexpr int kStep = kThreads / kVecs;
    const int di = kStep / rows, dx = kStep % rows;
    int i = (int)threadIdx.x / kVecs / rows, x = (int)threadIdx.x / kVecs % rows;
    while (i < n) {
        uint32_t par[kAhead];
        uint2 codes[kAhead];
        uint4 *dst[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int page = i < n ? s_page[i] : -2;
            par[u] = 0;
            codes[u] = make_uint2(0, 0);
            dst[u] = page == -2 ? nullptr
                                : reinterpret_cast<uint4 *>((x & 1 ? V : K) + ((size_t)(t0 + i) * Hkv + (x >> 1)) * D) + j;
            if (page >= 0) {
                const size_t row = ((size_t)page * Hkv + (x >> 1)) * a.page_size + s_off[i];
                const uint8_t *src = (x & 1 ? c.v_codes : c.k_codes) + row * (D * BITS / 8);
                par[u] = __ldg(reinterpret_cast<const uint32_t *>(x & 1 ? c.v_par : c.k_par) + row);
                if (BITS == 4) codes[u].x = __ldg(reinterpret_cast<const uint32_t *>(src) + j);
                else codes[u] = __ldg(reinterpret_cast<const uint2 *>(src) + j);
            }
            i += di;
            x += dx;
            if (x >= rows) {
                x -= rows;
                ++i;
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            // (an absent page: codes and parameters 0, so zeros)
            if (dst[u]) *dst[u] = BITS == 4 ? expand4(codes[u].x, par[u], e4)
                                            : expand8(codes[u].x, codes[u].y, par[u], e6);
        }
    }
}

// Tokens per CTA: several once the grid fills the GPU anyway.  Appends of 8192 tokens (48 heads) 48 us with four against
// 59 with one, of 2368 16 against 19, of 1200 13 against 12, of 64 10 against 6.
int tokens_per_cta(int T)
{
    return T >= 4 * 148 * kMaxTok ? kMaxTok : 1;
}

}  // namespace

cudaError_t launch_rotary(const uint16_t *x, int64_t ldx, const int32_t *pos, const AttnRotary &r, int T, int H, int d,
                          uint16_t *y, int64_t ldy, cudaStream_t stream)
{
    const int tb = tokens_per_cta(T);
    auto kernel = r.interleaved ? rotary_kernel<true> : rotary_kernel<false>;
    kernel<<<(T + tb - 1) / tb, kThreads, tb * (r.rot / 2) * (sizeof(double2) + sizeof(float2)), stream>>>(x, ldx, pos, r, T, H, d, tb, y, ldy);
    return cudaGetLastError();
}

cudaError_t launch_cache_append(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const uint16_t *q,
                                int64_t ldq, uint16_t *q_out, int64_t ldqo, int T, int Hq, int Hkv, int d,
                                const AttnRotary &r, const AttnCache &c, const AttnBatch &a, cudaStream_t stream)
{
    const int tb = tokens_per_cta(T);
    auto run = [&](auto kernel) {
        kernel<<<(T + tb - 1) / tb, kThreads, 0, stream>>>(k, ldk, v, ldv, q, ldq, q_out, ldqo, T, Hq, Hkv, r, c, a, tb);
    };
    auto pick = [&](auto half, auto inter) { r.interleaved ? run(inter) : run(half); };
    if (d == 128) c.bits == 4 ? pick(cache_append_kernel<128, 4, false>, cache_append_kernel<128, 4, true>)
                              : pick(cache_append_kernel<128, 8, false>, cache_append_kernel<128, 8, true>);
    else c.bits == 4 ? pick(cache_append_kernel<64, 4, false>, cache_append_kernel<64, 4, true>)
                     : pick(cache_append_kernel<64, 8, false>, cache_append_kernel<64, 8, true>);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const AttnCache &c, const AttnBatch &a, int T, int Hkv, int d, uint16_t *K, uint16_t *V,
                              cudaStream_t stream)
{
    // eight vectors per thread, as long as that leaves four CTAs per SM
    const int want = 8 * kThreads / (2 * Hkv * (d / 8)), most = T / (4 * 148);
    const int tb = std::max(1, std::min({want, most, kMaxReadTok}));
    auto run = [&](auto kernel) { kernel<<<(T + tb - 1) / tb, kThreads, 0, stream>>>(c, a, T, Hkv, tb, 0x64006400u, 0x54006400u, K, V); };
    if (d == 128) c.bits == 4 ? run(cache_read_kernel<128, 4>) : run(cache_read_kernel<128, 8>);
    else c.bits == 4 ? run(cache_read_kernel<64, 4>) : run(cache_read_kernel<64, 8>);
    return cudaGetLastError();
}

}  // namespace qoq
