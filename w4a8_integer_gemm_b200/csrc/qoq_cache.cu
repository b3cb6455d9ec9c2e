// qoq_cache.cu -- rotary positions, the paged 4/8-bit key/value cache's
// writer (with the rotation fused in) and its reader.
//
// All three move rows of heads once and are bound by HBM.  A "slot" is the
// unit of work: one thread, 16 channels of a head row in two 16-byte
// vectors chosen so that the thread holds both channels of its 8 rotation
// pairs: slot j takes pairs 8j .. 8j + 7, i.e. vectors j and j + rot/16
// (half layout) or 2j and 2j + 1 (interleaved, and the channels from rot
// on).  d / 16 neighbouring lanes make a head row, so the row's minimum and
// maximum for the quantiser are shuffles away.
//
// A rotation is computed in FP64 and rounded to FP16 once.  FP32 angles are
// off by up to pos * freq * 2^-24 (0.06 rad at position 2^20), and an FP32
// rotation lands on the wrong side of an FP16 rounding boundary about once
// in 4000 values, which would make the fused writer's codes differ from a
// rotation followed by a write.  sincospi of the angle's fraction of a turn
// needs no range reduction.
#include <cuda_fp16.h>

#include <cstdint>

#include "qoq_attn_internal.h"
#include "qoq_quant.cuh"

namespace qoq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;          // tokens per CTA
constexpr int kMaxPairs = 256;      // rot / 2 <= 256

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

__device__ __forceinline__ void unpack8(const uint4 &v, __half (&h)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[2 * i] = __ushort_as_half((uint16_t)(w[i] & 0xFFFFu));
        h[2 * i + 1] = __ushort_as_half((uint16_t)(w[i] >> 16));
    }
}

__device__ __forceinline__ uint4 pack8(const __half (&h)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)__half_as_ushort(h[2 * i]) | ((uint32_t)__half_as_ushort(h[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void rotate_pair(__half &a, __half &b, double2 cs)
{
    const double x1 = (double)__half2float(a), x2 = (double)__half2float(b);
    a = __double2half(fma(x1, cs.x, -(x2 * cs.y)));
    b = __double2half(fma(x1, cs.y, x2 * cs.x));
}

// Rotates the 8 pairs of a slot (a, b: its two vectors) by cs[0..7].
__device__ __forceinline__ void rotate_slot(__half (&a)[8], __half (&b)[8], const double2 *cs, int interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate_pair(a[2 * i], a[2 * i + 1], cs[i]);
            rotate_pair(b[2 * i], b[2 * i + 1], cs[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate_pair(a[i], b[i], cs[i]);
    }
}

// ---------------------------------------------------------------- rotary --
__global__ void __launch_bounds__(kThreads) rotary_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                                                          const int32_t *__restrict__ pos, AttnRotary r, int T, int H,
                                                          int d, int tb, uint16_t *y, int64_t ldy)
{
    __shared__ double2 cs[kMaxTok][kMaxPairs];
    const int t0 = blockIdx.x * tb, n = min(tb, T - t0), pairs = r.rot / 2;
    for (int e = threadIdx.x; e < n * pairs; e += kThreads)
        cs[e / pairs][e % pairs] = turn(__ldg(pos + t0 + e / pairs), __ldg(r.freq + e % pairs), r.amplitude);
    __syncthreads();
    const int slots = d / 16;
    for (int e = threadIdx.x; e < n * H * slots; e += kThreads) {
        const int j = e % slots, h = e / slots % H, i = e / (slots * H);
        const int2 at = slot_vectors(j, r.rot, r.interleaved);
        const uint4 *src = reinterpret_cast<const uint4 *>(x + (t0 + i) * ldx + (size_t)h * d);
        uint4 *dst = reinterpret_cast<uint4 *>(y + (t0 + i) * ldy + (size_t)h * d);
        uint4 va = src[at.x], vb = src[at.y];
        if (j < r.rot / 16) {
            __half a[8], b[8];
            unpack8(va, a);
            unpack8(vb, b);
            rotate_slot(a, b, &cs[i][8 * j], r.interleaved);
            va = pack8(a);
            vb = pack8(b);
        }
        dst[at.x] = va;
        dst[at.y] = vb;
    }
}

// ---------------------------------------------------------------- append --
__device__ __forceinline__ uint32_t code_of(float x, float m, float s, float top)
{
    return s == 0.0f ? 0u : (uint32_t)(int)fminf(rintf(__fdiv_rn(x - m, s)), top);
}

// Codes of the 8 channels of a vector, channel 0 lowest.
template <int BITS>
__device__ __forceinline__ uint64_t codes8(const __half (&h)[8], float m, float s)
{
    uint64_t o = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o |= (uint64_t)code_of(__half2float(h[i]), m, s, (float)((1 << BITS) - 1)) << (BITS * i);
    return o;
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(
    const uint16_t *__restrict__ k, int64_t ldk, const uint16_t *__restrict__ v, int64_t ldv, const uint16_t *q,
    int64_t ldq, uint16_t *q_out, int64_t ldqo, int T, int Hq, int Hkv, AttnRotary r, AttnCache c, AttnBatch a, int tb)
{
    constexpr int kSlots = D / 16;
    __shared__ double2 cs[kMaxTok][D / 2];
    __shared__ int s_pos[kMaxTok], s_page[kMaxTok];
    const int t0 = blockIdx.x * tb, n = min(tb, T - t0), pairs = r.rot / 2;
    if (threadIdx.x < n) {
        const int t = t0 + threadIdx.x, b = sequence_of(a.cu, a.B, t);
        const int pos = b < 0 ? 0 : __ldg(a.kv_len + b) - (__ldg(a.cu + b + 1) - t);
        s_pos[threadIdx.x] = pos;
        s_page[threadIdx.x] = b < 0 ? -2 : page_of(a, b, pos);   // -2: no sequence
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n * pairs; e += kThreads)
        cs[e / pairs][e % pairs] = turn(s_pos[e / pairs], __ldg(r.freq + e % pairs), r.amplitude);
    __syncthreads();
    const int H = Hq + 2 * Hkv;     // head rows of a token: q, then k, then v
    const int items = n * H * kSlots;
    // every lane takes part in the shuffles of each pass; lanes past the end do nothing else
    for (int e0 = 0; e0 < items; e0 += kThreads) {
        const int e = e0 + threadIdx.x;
        const bool in = e < items;
        const int j = e % kSlots, h = e / kSlots % H, i = in ? e / (kSlots * H) : 0;
        const int page = s_page[i];
        const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hkv;
        const bool work = in && page != -2 && (is_q || page >= 0);
        const int rot = is_q || is_k ? r.rot : 0;
        const int2 at = slot_vectors(j, rot, r.interleaved);
        __half x[8], y[8];
        float lo = 0.0f, hi = 0.0f;
        if (work) {
            const int t = t0 + i;
            const uint16_t *row = is_q ? q + t * ldq + (size_t)h * D
                                  : is_k ? k + t * ldk + (size_t)(h - Hq) * D
                                         : v + t * ldv + (size_t)(h - Hq - Hkv) * D;
            unpack8(reinterpret_cast<const uint4 *>(row)[at.x], x);
            unpack8(reinterpret_cast<const uint4 *>(row)[at.y], y);
            if (j < rot / 16) rotate_slot(x, y, &cs[i][8 * j], r.interleaved);
            if (is_q) {
                uint4 *dst = reinterpret_cast<uint4 *>(q_out + t * ldqo + (size_t)h * D);
                dst[at.x] = pack8(x);
                dst[at.y] = pack8(y);
            } else {
                lo = hi = __half2float(x[0]);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float f = __half2float(x[u]), g = __half2float(y[u]);
                    lo = fminf(lo, fminf(f, g));
                    hi = fmaxf(hi, fmaxf(f, g));
                }
            }
        }
#pragma unroll
        for (int o = 1; o < kSlots; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (work && !is_q) {
            const __half sh = __float2half_rz(__fdiv_rn(hi - lo, (float)((1 << BITS) - 1)));
            const float s = __half2float(sh);
            const int hk = is_k ? h - Hq : h - Hq - Hkv;
            const size_t row = ((size_t)page * Hkv + hk) * a.page_size + (s_pos[i] & (a.page_size - 1));
            uint8_t *dst = (is_k ? c.k_codes : c.v_codes) + row * (D * BITS / 8);
            const uint64_t cx = codes8<BITS>(x, lo, s), cy = codes8<BITS>(y, lo, s);
            if (BITS == 4) {
                reinterpret_cast<uint32_t *>(dst)[at.x] = (uint32_t)cx;
                reinterpret_cast<uint32_t *>(dst)[at.y] = (uint32_t)cy;
            } else {
                reinterpret_cast<uint64_t *>(dst)[at.x] = cx;
                reinterpret_cast<uint64_t *>(dst)[at.y] = cy;
            }
            if (j == 0)
                reinterpret_cast<uint32_t *>(is_k ? c.k_par : c.v_par)[row] =
                    (uint32_t)__half_as_ushort(sh) | ((uint32_t)float_to_half_bits(lo) << 16);
        }
    }
}

// ------------------------------------------------------------------ read --
// fp16(s * c + m): the half-precision multiply-add rounds once.
template <int BITS>
__device__ __forceinline__ uint4 values8(uint64_t codes, uint32_t par)
{
    const __half2 s = __half2half2(__ushort_as_half((uint16_t)(par & 0xFFFFu)));
    const __half2 m = __half2half2(__ushort_as_half((uint16_t)(par >> 16)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c0 = (uint32_t)(codes >> (2 * i * BITS)) & ((1u << BITS) - 1);
        const uint32_t c1 = (uint32_t)(codes >> ((2 * i + 1) * BITS)) & ((1u << BITS) - 1);
        // 1024 + c in FP16 has c as its low mantissa bits
        const uint32_t u = (c0 | (c1 << 16)) | 0x64006400u;
        const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&u), __half2half2(__ushort_as_half(0x6400)));
        const __half2 x = __hfma2(c, s, m);
        w[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(AttnCache c, AttnBatch a, int T, int Hkv, int tb,
                                                              uint16_t *__restrict__ K, uint16_t *__restrict__ V)
{
    constexpr int kVecs = D / 8;
    __shared__ int s_off[kMaxTok], s_page[kMaxTok];
    const int t0 = blockIdx.x * tb, n = min(tb, T - t0);
    if (threadIdx.x < n) {
        const int t = t0 + threadIdx.x, b = sequence_of(a.cu, a.B, t);
        const int pos = b < 0 ? 0 : __ldg(a.kv_len + b) - (__ldg(a.cu + b + 1) - t);
        s_page[threadIdx.x] = b < 0 ? -2 : page_of(a, b, pos);
        s_off[threadIdx.x] = pos & (a.page_size - 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n * 2 * Hkv * kVecs; e += kThreads) {
        const int j = e % kVecs, h = e / kVecs % Hkv, val = e / (kVecs * Hkv) & 1, i = e / (kVecs * Hkv * 2);
        const int page = s_page[i];
        if (page == -2) continue;
        uint4 o = make_uint4(0, 0, 0, 0);
        if (page >= 0) {
            const size_t row = ((size_t)page * Hkv + h) * a.page_size + s_off[i];
            const uint8_t *src = (val ? c.v_codes : c.k_codes) + row * (D * BITS / 8);
            const uint32_t par = __ldg(reinterpret_cast<const uint32_t *>(val ? c.v_par : c.k_par) + row);
            const uint64_t codes = BITS == 4 ? (uint64_t)__ldg(reinterpret_cast<const uint32_t *>(src) + j)
                                             : (uint64_t)__ldg(reinterpret_cast<const unsigned long long *>(src) + j);
            o = values8<BITS>(codes, par);
        }
        reinterpret_cast<uint4 *>((val ? V : K) + ((size_t)(t0 + i) * Hkv + h) * D)[j] = o;
    }
}

// Tokens per CTA: several once the grid fills the GPU anyway.
int tokens_per_cta(int T)
{
    return T >= 4 * 148 * kMaxTok ? kMaxTok : 1;
}

}  // namespace

cudaError_t launch_rotary(const uint16_t *x, int64_t ldx, const int32_t *pos, const AttnRotary &r, int T, int H, int d,
                          uint16_t *y, int64_t ldy, cudaStream_t stream)
{
    const int tb = tokens_per_cta(T);
    rotary_kernel<<<(T + tb - 1) / tb, kThreads, 0, stream>>>(x, ldx, pos, r, T, H, d, tb, y, ldy);
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
    if (d == 128) c.bits == 4 ? run(cache_append_kernel<128, 4>) : run(cache_append_kernel<128, 8>);
    else c.bits == 4 ? run(cache_append_kernel<64, 4>) : run(cache_append_kernel<64, 8>);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const AttnCache &c, const AttnBatch &a, int T, int Hkv, int d, uint16_t *K, uint16_t *V,
                              cudaStream_t stream)
{
    const int tb = tokens_per_cta(T);
    auto run = [&](auto kernel) { kernel<<<(T + tb - 1) / tb, kThreads, 0, stream>>>(c, a, T, Hkv, tb, K, V); };
    if (d == 128) c.bits == 4 ? run(cache_read_kernel<128, 4>) : run(cache_read_kernel<128, 8>);
    else c.bits == 4 ? run(cache_read_kernel<64, 4>) : run(cache_read_kernel<64, 8>);
    return cudaGetLastError();
}

}  // namespace qoq
