// qoq_attn_tile.cu -- attention in tiles of 256 rows x 128 keys on the
// tensor cores (tcgen05): whole prompts (FP16 keys and values), and chunks
// of new tokens over the paged 4/8-bit cache.
//
// Mathematics: one pass over the keys with the running maximum and sum of
// the softmax, O = sum_j exp(s_j - m) v_j, out = O / sum_j exp(s_j - m).
//
// A CTA owns 256 rows of one sequence and KV head: row = (new token, query
// head of the group), so the heads that share a KV head share its tiles and
// any group size fills the tile.  Two row tiles of 128 are in flight: while
// one's softmax runs on the CUDA cores the tensor cores work for the other.
//   warps 0-3, 4-7   softmax of row tile 0 and 1, one row per thread: S from
//                    tensor memory, masks, maximum, exp2, P as FP16 back to
//                    tensor memory over S; rescale O (tensor memory) when
//                    the maximum grew by more than 2^8; at the end O to HBM.
//   warps 8-11       loader: keys and values of the tile into a ring of
//                    shared-memory slots in the 128-byte-swizzled layout:
//                    cp.async for FP16 rows, or the codes expanded to
//                    fp16(s c + m) in registers.
//   warp 12          one thread issues the MMAs: S = Q K^T (both from shared
//                    memory), O += P V (P from tensor memory, V with its
//                    channels contiguous).
// Tensor memory: S0 S1 (128 columns each, P over the first half), O0 O1 (D
// columns each).
//
// Roundings below FP32: P (FP16, as the tensor core's operand: half a step of
// each weight; the sum of weights is taken before it, in FP32) and, for a
// cache, the expanded keys and values (half a step, against a quantisation
// step of 1/15 or 1/255 of the row's range).
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "qoq_attn_internal.h"
#include "qoq_attn_device.cuh"
#include "qoq_ptx.cuh"
#include "qoq_quant.cuh"

namespace qoq {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 256;          // rows of a CTA (two tiles of 128)
constexpr int kKeys = 128;          // keys of a tile
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr uint64_t kBudgetNs = 2000000000ull;

__device__ int g_tile_error;        // non-zero after a bounded wait ran out

template <int D>
struct TileCfg {
    static constexpr int kBlock = kKeys * 128;              // [128 rows][64 channels] FP16, swizzled
    static constexpr int kTile = kBlock * (D / 64);         // K, V or Q of 128 rows
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr int kQ = 0;                            // two Q tiles
    static constexpr int kRing = 2 * kTile;
    static constexpr int kBars = kRing + kSlots * kTile;
    static constexpr int kSmem = kBars + 256 + 1024;        // + alignment
};

struct TileArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv, ldo;
    uint16_t *out;
    float *part;            // [splits][T * Hq][D] sums and, after them, [splits][T * Hq][2] (maximum, sum); null: no split
    AttnCache c;
    AttnBatch a;
    int T, Hq, Hkv, G, splits;
    int few;                // sequences with at most this many rows (n_b * G) are another kernel's
    float scale_log2;       // |scale| * log2(e)
    uint32_t flip;          // 0x80008000 when scale < 0: the sign goes into q
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two FP32 numbers in a register pair, and the instructions that work on both.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// byte offset of 16-byte vector `vec` of row `row` in a [rows][64 channels] block, 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int row, int vec)
{
    return (uint32_t)(row * 128 + (((vec & 7) ^ (row & 7)) << 4));
}

template <int N>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Registers: launched with 512 x 128; 2 x 128 x 184 + 128 x 96 + 128 x 48 = 512 x 128.
constexpr int kRegsSoftmax = 184, kRegsLoader = 96, kRegsMma = 48;
static_assert(256 * kRegsSoftmax + 128 * kRegsLoader + 128 * kRegsMma <= kThreads * 128, "register split");

// BITS 0: FP16 rows of the batch itself (prompts); 4 or 8: the cache.
template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) attn_tile_kernel(const TileArgs p)
{
    using C = TileCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ TileScan scan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int hk = id % p.Hkv;

    // ---- which rows, which keys ----
    const TileWork w = find_tile(p.a, p.T, p.G, kRows, p.few + 1, 1 << 30, id / p.Hkv, scan);
    if (w.b < 0) return;
    const int n = w.n, rows = n * p.G - w.row0;                      // rows of the sequence from this tile on
    const int first = BITS ? __ldg(p.a.kv_len + w.b) - n : 0;        // position of its new token 0
    const int t_seq = __ldg(p.a.cu + w.b);                           // its first row
    // keys seen by the last row of each row tile, in key tiles
    int last[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int r = min(rows, 128 * (t + 1)) - 1;
        last[t] = rows > 128 * t ? max(0, first + (w.row0 + r) / p.G + 1) : 0;
        if (BITS) last[t] = min(last[t], p.a.table_pages * p.a.page_size);
    }
    const int all = (max(last[0], last[1]) + kKeys - 1) / kKeys;
    const int j0 = (int)((int64_t)all * split / p.splits), j1 = (int)((int64_t)all * (split + 1) / p.splits);
    int cnt[2];                                                      // key tiles of each row tile here
#pragma unroll
    for (int t = 0; t < 2; ++t) cnt[t] = max(0, min((last[t] + kKeys - 1) / kKeys, j1) - j0);
    const int steps = max(cnt[0], cnt[1]);

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_addr(smem);
    const uint32_t bars = sbase + C::kBars;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (C::kSlots + s); };
    auto sfull = [&](int t) { return bars + 8u * (2 * C::kSlots + t); };
    auto pfull = [&](int t) { return bars + 8u * (2 * C::kSlots + 2 + t); };
    auto ofull = [&](int t) { return bars + 8u * (2 * C::kSlots + 4 + t); };
    const uint32_t done = bars + 8u * (2 * C::kSlots + 6);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(full(s), 4);
            mbar_init(empty(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(sfull(t), 1);
            mbar_init(pfull(t), 4);
            mbar_init(ofull(t), 1);
        }
        mbar_init(done, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(smem_addr(&tmem_slot), 512);
        tmem_relinquish();
    }
    // ---- Q: 256 rows into shared memory, zeros past the end ----
    if (steps > 0) {
        for (int e = threadIdx.x; e < kRows * (D / 8); e += kThreads) {
            const int r = e / (D / 8), vec = e % (D / 8);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int tok = (w.row0 + r) / p.G, g = (w.row0 + r) % p.G;
                x = __ldg(reinterpret_cast<const uint4 *>(p.q + (int64_t)(t_seq + tok) * p.ldq +
                                                          (size_t)(hk * p.G + g) * D) + vec);
                x = make_uint4(x.x ^ p.flip, x.y ^ p.flip, x.z ^ p.flip, x.w ^ p.flip);
                if (BITS == 4) x = to_code_order(x);
            }
            *reinterpret_cast<uint4 *>(smem + C::kQ + (r >> 7) * C::kTile + (vec >> 3) * C::kBlock + swz(r & 127, vec)) = x;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp >= 12) {
        // ------------------------------------------------------------ MMA --
        regs_down<kRegsMma>();
        if (warp == 12 && lane == 0 && steps > 0) {
            const uint32_t is = idesc_f16_m128(kKeys, false), io = idesc_f16_m128(D, true);
            auto scores = [&](int t, int slot) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * C::kBlock;
                    const uint64_t qa = smem_desc_sw128(sbase + C::kQ + t * C::kTile + off) + 2 * (kk & 3);
                    const uint64_t kb = smem_desc_sw128(sbase + C::kRing + slot * C::kTile + off) + 2 * (kk & 3);
                    mma_f16_ss(tmem + 128 * t, qa, kb, is, kk > 0);
                }
                mma_commit(sfull(t));
            };
            auto values = [&](int t, int slot, bool accumulate) {
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk) {
                    const uint64_t vb = smem_desc_sw128_mn(sbase + C::kRing + slot * C::kTile + kk * 2048, C::kBlock);
                    mma_f16_ts(tmem + 256 + D * t, tmem + 128 * t + 8 * kk, vb, io, accumulate || kk > 0);
                }
            };
            // ring items: K of step i is item 2i, V is item 2i + 1
            auto ready = [&](int item) {
                return wait_short(full(item % C::kSlots), (uint32_t)(item / C::kSlots) & 1, &abort_flag, kBudgetNs);
            };
            bool ok = ready(0);
            if (ok) {
                tc_fence_after();
                for (int t = 0; t < 2; ++t)
                    if (cnt[t] > 0) scores(t, 0);
                mma_commit(empty(0));
            }
            for (int i = 0; i < steps && ok; ++i) {
                const int vi = 2 * i + 1, ki = 2 * i + 2;
                ok = ready(vi) && (i + 1 >= steps || ready(ki));
                for (int t = 0; t < 2 && ok; ++t) {
                    if (i >= cnt[t]) continue;
                    ok = wait_short(pfull(t), (uint32_t)i & 1, &abort_flag, kBudgetNs);
                    if (!ok) break;
                    tc_fence_after();
                    values(t, vi % C::kSlots, i > 0);
                    // S of the next step goes over P of this one: MMAs run in the order they were issued
                    if (i + 1 < cnt[t]) scores(t, ki % C::kSlots);
                    else mma_commit(ofull(t));
                }
                if (!ok) break;
                mma_commit(empty(vi % C::kSlots));
                if (i + 1 < steps) mma_commit(empty(ki % C::kSlots));
            }
            if (!ok) {      // let what was issued finish before tensor memory is freed
                mma_commit(done);
                const uint64_t end = global_timer_ns() + 200000000ull;
                while (!mbar_try_wait(done, 0) && global_timer_ns() < end) {
                }
            }
        }
    } else if (warp >= 8) {
        // --------------------------------------------------------- loader --
        regs_down<kRegsLoader>();
        const int tid = threadIdx.x - 256;
        const int items = 2 * steps;
        auto slot_free = [&](int item) {
            if (item < C::kSlots) return true;
            return (bool)__all_sync(0xffffffffu, wait_short(empty(item % C::kSlots), (uint32_t)(item / C::kSlots - 1) & 1,
                                                              &abort_flag, kBudgetNs));
        };
        auto signal = [&](int item) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(item % C::kSlots));
        };
        if (BITS == 0) {
            constexpr int kVecs = D / 8, kPass = 128 / kVecs;        // rows a pass of the 128 threads covers: 8 or 16,
                                                                     // so the swizzle of a thread's rows is one number
            constexpr int kLag = 2;                                  // items in flight behind the newest
            const int vec = tid % kVecs, r0 = tid / kVecs;
            const uint32_t my_dst = sbase + C::kRing + (vec >> 3) * C::kBlock + swz(r0, vec);
            const uint16_t *kp = p.k + (int64_t)(t_seq + j0 * kKeys + r0) * p.ldk + (size_t)hk * D + vec * 8;
            const uint16_t *vp = p.v + (int64_t)(t_seq + j0 * kKeys + r0) * p.ldv + (size_t)hk * D + vec * 8;
            const int64_t k_pass = p.ldk * kPass, v_pass = p.ldv * kPass;
            bool ok = true;
            for (int item = 0; item < items + kLag; ++item) {
                if (item < items) {
                    ok = slot_free(item);
                    if (!ok) break;
                    const bool val = item & 1;
                    const int left = n - (j0 + (item >> 1)) * kKeys - r0;    // rows past the sequence are zeros
                    const uint16_t *src = val ? vp : kp;
                    const int64_t pass = val ? v_pass : k_pass;
                    const uint32_t dst = my_dst + (item % C::kSlots) * C::kTile;
                    if (left >= kKeys - r0) {
#pragma unroll
                        for (int i = 0; i < kKeys / kPass; ++i, src += pass) cp_async<16>(dst + i * kPass * 128, src);
                    } else {
#pragma unroll 4
                        for (int i = 0; i < kKeys / kPass; ++i, src += pass)
                            cp_async16(dst + i * kPass * 128, i * kPass < left ? src : p.k, i * kPass < left);
                    }
                    (val ? vp : kp) += (val ? p.ldv : p.ldk) * kKeys;
                }
                cp_async_commit();
                if (item >= kLag) {
                    cp_async_wait<kLag>();
                    signal(item - kLag);
                }
            }
            cp_async_wait<0>();
        } else {
            // Lanes share a row's bytes, 16 each; a thread's rows are kPass apart.
            constexpr int kB = BITS ? BITS : 4;
            constexpr int kRowBytes = D * kB / 8, kLanes = kRowBytes / 16, kPass = 128 / kLanes, kN = kKeys / kPass;
            const int part = tid % kLanes, r0 = tid / kLanes;
            uint4 kc[kN], vc[kN];
            uint32_t kp[kN], vp[kN];
            uint32_t at[kN];                                         // cache row of the thread's keys (a pool of 2^32 rows
                                                                     // would not fit the GPU), or kNone
            auto locate = [&](int step) {
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const int pos = (j0 + step) * kKeys + r0 + i * kPass;
                    const int page = pos < first + n ? page_of(p.a, w.b, pos) : -1;
                    at[i] = page < 0 ? kNone
                                     : ((uint32_t)page * p.Hkv + hk) * p.a.page_size + (pos & (p.a.page_size - 1));
                }
            };
            auto fetch = [&](uint4 (&c)[kN], uint32_t (&pr)[kN], const uint8_t *codes, const uint16_t *par) {
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    c[i] = make_uint4(0, 0, 0, 0);
                    pr[i] = 0;
                    if (at[i] != kNone) {
                        c[i] = __ldg(reinterpret_cast<const uint4 *>(codes + (size_t)at[i] * kRowBytes) + part);
                        pr[i] = __ldg(reinterpret_cast<const uint32_t *>(par) + at[i]);
                    }
                }
            };
            auto expand = [&](int item, const uint4 (&c)[kN], const uint32_t (&pr)[kN]) {
                uint8_t *dst = smem + C::kRing + (item % C::kSlots) * C::kTile;
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const int r = r0 + i * kPass;
                    const uint32_t cw[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
                    if (kB == 4) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            // the upper lanes of a row store in another order: eight lanes, eight bank groups
                            const bool other = D == 128 && (part & 2);
                            const int vec = 4 * part + (other ? u ^ 2 : u);
                            *reinterpret_cast<uint4 *>(dst + (vec >> 3) * C::kBlock + swz(r, vec)) =
                                expand4(other ? cw[u ^ 2] : cw[u], pr[i]);
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const bool other = D == 128 && (part & 4);
                            const int vec = 2 * part + (other ? u ^ 1 : u);
                            *reinterpret_cast<uint4 *>(dst + (vec >> 3) * C::kBlock + swz(r, vec)) =
                                expand8(other ? cw[2 * (u ^ 1)] : cw[2 * u], other ? cw[2 * (u ^ 1) + 1] : cw[2 * u + 1], pr[i]);
                        }
                    }
                }
            };
            if (steps > 0) {
                locate(0);
                fetch(kc, kp, p.c.k_codes, p.c.k_par);
                fetch(vc, vp, p.c.v_codes, p.c.v_par);
            }
            for (int i = 0; i < steps; ++i) {
                if (i + 1 < steps) locate(i + 1);
                if (!slot_free(2 * i)) break;
                expand(2 * i, kc, kp);
                signal(2 * i);
                if (i + 1 < steps) fetch(kc, kp, p.c.k_codes, p.c.k_par);
                if (!slot_free(2 * i + 1)) break;
                expand(2 * i + 1, vc, vp);
                signal(2 * i + 1);
                if (i + 1 < steps) fetch(vc, vp, p.c.v_codes, p.c.v_par);
            }
        }
    } else {
        // -------------------------------------------------------- softmax --
        regs_up<kRegsSoftmax>();
        const int t = warp >> 2, r = (warp & 3) * 32 + lane;         // row tile, row of it
        const int row = 128 * t + r;                                 // of the CTA
        const bool real = row < rows;
        const int tok = real ? (w.row0 + row) / p.G : 0, g = real ? (w.row0 + row) % p.G : 0;
        const int see = real ? first + tok + 1 : 0;                  // keys 0 .. see - 1 are seen
        const int see_min = __reduce_min_sync(0xffffffffu, see);
        const uint32_t ts = tmem + 128 * t + ((uint32_t)(warp & 3) << 21);
        const uint32_t to = tmem + 256 + D * t + ((uint32_t)(warp & 3) << 21);
        const float sl = p.scale_log2;
        float m = -INFINITY, l = 0.0f;                               // maximum in use (log2 units), sum
        bool ok = true;
        for (int i = 0; i < cnt[t]; ++i) {
            const int key0 = (j0 + i) * kKeys;
            // (cache) which 16-token pieces of the tile are there
            uint32_t there = 0xFFu;
            if (BITS) there = __ballot_sync(0xffffffffu, lane < 8 && page_of(p.a, w.b, key0 + 16 * lane) >= 0);
            ok = __all_sync(0xffffffffu, wait_short(sfull(t), (uint32_t)i & 1, &abort_flag, kBudgetNs));
            if (!ok) break;
            tc_fence_after();
            const int lim = see - key0;
            auto softmax = [&](auto masked) {
                // -inf over the columns [c0, c0 + n) of x that the row does not see
                auto mask = [&](uint32_t *x, int c0, int n) {
#pragma unroll
                    for (int c = 0; c < n; ++c)
                        if (c0 + c >= lim || !((there >> ((c0 + c) >> 4)) & 1)) x[c] = 0xFF800000u;
                };
                // pass 1: the row's maximum.  S is read from tensor memory twice, 32 columns at a time (a read costs
                // little, and a whole row in registers costs moves and spills)
                float top = -INFINITY;
#pragma unroll
                for (int c0 = 0; c0 < kKeys; c0 += 64) {
                    uint32_t x[64];
                    tmem_ld32x2(ts + c0, ts + c0 + 32, x, x + 32);
                    if (masked.value) mask(x, c0, 64);
                    float mx[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 64; c += 2)
                        mx[c / 2 & 3] = fmaxf(fmaxf(mx[c / 2 & 3], __uint_as_float(x[c])), __uint_as_float(x[c + 1]));
                    top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                }
                top *= sl;
                // The maximum in use lags behind by up to 2^8: weights stay below 2^8 (FP16 holds 2^15), and O is
                // rescaled rarely instead of in every tile.
                const bool grow = top > m + 8.0f || (m == -INFINITY && top > -INFINITY);
                if (__any_sync(0xffffffffu, grow)) {
                    const float m1 = grow ? top : m;
                    const float keep = m == -INFINITY ? 0.0f : ex2(m - m1);
                    m = m1;
                    l *= keep;
                    if (i > 0) {
                        // S of this step is complete, so is P V of the last one (issued before it)
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(to + c, o);
#pragma unroll
                            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * keep);
                            tmem_st32(to + c, o);
                        }
                    }
                }
                // pass 2: P = 2^(s - m), FP16, over the columns of S already read
                const float sub = m == -INFINITY ? 0.0f : -m;
                const uint64_t sl2 = pair(sl, sl), sub2 = pair(sub, sub);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c0 = 0; c0 < kKeys; c0 += 32) {
                    uint32_t x[32], pk[16];
                    tmem_ld32(ts + c0, x);
                    if (masked.value) mask(x, c0, 32);
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        float a, b;
                        unpair(fma2(pair(__uint_as_float(x[2 * u]), __uint_as_float(x[2 * u + 1])), sl2, sub2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[u & 1] = add2(sum[u & 1], pair(a, b));
                        const __half2 h = __floats2half2_rn(a, b);
                        pk[u] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    tmem_st16(ts + c0 / 2, pk);
                }
                float a, b;
                unpair(add2(sum[0], sum[1]), a, b);
                l += a + b;
            };
            if (see_min < key0 + kKeys || there != 0xFFu) softmax(std::true_type{});
            else softmax(std::false_type{});
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull(t));
        }
        // ---- O out ----
        if (ok && cnt[t] > 0) {
            ok = __all_sync(0xffffffffu, wait_short(ofull(t), 0, &abort_flag, kBudgetNs));
            tc_fence_after();
        }
        if (ok) {
            const int64_t orow = (int64_t)(t_seq + tok) * p.Hq + hk * p.G + g;
            if (p.part == nullptr) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                uint16_t *dst = p.out + (int64_t)(t_seq + tok) * p.ldo + (size_t)(hk * p.G + g) * D;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    if (cnt[t] > 0) tmem_ld32(to + c, o);
                    uint32_t h[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        const __half2 x = __floats2half2_rn(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv);
                        h[u] = l > 0.0f ? *reinterpret_cast<const uint32_t *>(&x) : 0u;
                    }
                    if (real) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint4 x = make_uint4(h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
                            if (BITS == 4) x = from_code_order(x);
                            reinterpret_cast<uint4 *>(dst)[c / 8 + u] = x;
                        }
                    }
                }
            } else {
                const int64_t all_rows = (int64_t)p.T * p.Hq;
                float *dst = p.part + ((int64_t)split * all_rows + orow) * D;
                if (real) {
                    float2 *ml = reinterpret_cast<float2 *>(p.part + (int64_t)p.splits * all_rows * D);
                    ml[(int64_t)split * all_rows + orow] = make_float2(m, l);
                }
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    if (cnt[t] > 0) {
                        tmem_ld32(to + c, o);
                        if (real && l > 0.0f) {
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                const uint32_t *x = o + 8 * (u >> 1);
                                // columns 8v .. 8v + 7 hold channels 0 4 1 5 2 6 3 7 of a 4-bit cache
                                uint4 y = make_uint4(x[4 * (u & 1)], x[4 * (u & 1) + 1], x[4 * (u & 1) + 2], x[4 * (u & 1) + 3]);
                                if (BITS == 4) y = make_uint4(x[u & 1], x[2 + (u & 1)], x[4 + (u & 1)], x[6 + (u & 1)]);
                                reinterpret_cast<uint4 *>(dst)[c / 4 + u] = y;
                            }
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && abort_flag) atomicExch(&g_tile_error, 1);
}

template <int D, int BITS>
cudaError_t launch_tile(const TileArgs &p, cudaStream_t stream)
{
    auto kernel = attn_tile_kernel<D, BITS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    // every sequence wastes at most one part of a row tile
    const int64_t tiles = (int64_t)p.T * p.G / kRows + (p.a.B < p.T ? p.a.B : p.T);
    kernel<<<(unsigned)(tiles * p.Hkv * p.splits), kThreads, TileCfg<D>::kSmem, stream>>>(p);
    return cudaGetLastError();
}

constexpr float kLog2e = 1.4426950408889634f;

void set_scale(TileArgs &p, float scale)
{
    // a zero scale keeps a tiny one: the same uniform weights, and no 0 * infinity at masked scores
    p.scale_log2 = fmaxf(fabsf(scale) * kLog2e, 1e-30f);
    p.flip = scale < 0.0f ? 0x80008000u : 0u;
}

}  // namespace

cudaError_t launch_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                                    int64_t ldv, int T, int Hq, int Hkv, int d, const AttnBatch &a, float scale,
                                    uint16_t *out, int64_t ldo, cudaStream_t stream)
{
    TileArgs p{q, k, v, ldq, ldk, ldv, ldo, out, nullptr, AttnCache{}, a, T, Hq, Hkv, Hq / Hkv, 1, 0, 0.0f, 0u};
    set_scale(p, scale);
    return d == 128 ? launch_tile<128, 0>(p, stream) : launch_tile<64, 0>(p, stream);
}

cudaError_t launch_paged_tiles(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                               const AttnBatch &a, int few, int splits, float scale, uint16_t *out, int64_t ldo,
                               float *part, cudaStream_t stream)
{
    TileArgs p{q, nullptr, nullptr, ldq, 0, 0, ldo, out, part, c, a, T, Hq, Hkv, Hq / Hkv, splits, few, 0.0f, 0u};
    set_scale(p, scale);
    if (d == 128) return c.bits == 4 ? launch_tile<128, 4>(p, stream) : launch_tile<128, 8>(p, stream);
    return c.bits == 4 ? launch_tile<64, 4>(p, stream) : launch_tile<64, 8>(p, stream);
}

cudaError_t read_and_clear_tile_error(int *value)
{
    *value = 0;
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tile_error, sizeof(int));
    if (e != cudaSuccess) return e;
    if (v) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_tile_error, &zero, sizeof(int));
    }
    *value = v;
    return e;
}

}  // namespace qoq
