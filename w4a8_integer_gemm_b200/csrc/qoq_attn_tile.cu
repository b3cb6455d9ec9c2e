// qoq_attn_tile.cu -- attention in tiles of 256 rows x 128 keys on the
// tensor cores (tcgen05): whole prompts (FP16 keys and values), and chunks
// of new tokens over the paged 4/8-bit cache.
//
// Mathematics: one pass over the keys with the running maximum and sum of
// the softmax, O = sum_j exp(s_j - m) v_j, out = O / sum_j exp(s_j - m).
//
// A work item is 256 rows of one sequence and KV head: row = (new token, query
// head of the group), so the heads that share a KV head share its tiles and
// any group size fills the tile.  Two row tiles of 128 are in flight: while
// one's softmax runs on the CUDA cores the tensor cores work for the other.
// One CTA per SM stays and works through a list of items:
//   warps 0-7, 8-15  softmax of row tile 0 and 1, two threads to a row: S from
//                    tensor memory, masks, exp2, P as FP16 back to tensor
//                    memory over S; now and then a new maximum, and O
//                    (tensor memory) rescaled; at the end O to HBM.
//   loaders          keys and values of the tile into a ring of shared-memory
//                    slots in the 128-byte-swizzled layout: a warp with TMA
//                    for FP16 rows; for a cache a warpgroup that expands
//                    the codes to fp16(s c + m) in registers.
//   MMA              S = Q K^T (both from shared memory), O += P V (P from
//                    tensor memory, V with its channels contiguous).
//   Q                the next item's Q as soon as the last S of this one is
//                    done.  (Boxes by TMA, where the group's heads divide
//                    128, were no faster: the softmax is not done earlier.)
//   plan             the list, a few items ahead, in a ring of descriptions.
// Tensor memory: S0 S1 (128 columns each, P over the first half), O0 O1 (D
// columns each).
//
// Lists.  Prompts: whole items, those that see most first, dealt to and fro
// over the CTAs.  A cache: the line of all (item, key tile) is cut into equal
// shares, one per CTA; an item that spans CTAs leaves a part in each, and a
// second kernel joins them.  (Whole items, and keys cut into equal numbers of
// tiles per item: chunks of 450 to 600 tokens over up to 13600 255 us against
// 235, a mixed batch of short chunks 94 us against 76, at that time.)
//
// Bound: for each row tile a step is a chain, softmax (about 1300 cycles of
// its 16 warps' exponentials and conversions, 900 of waits and stores) and
// then 1060 cycles of MMAs, one after the other: P lies over the first half of
// S, and the next S, a whole one, waits until P V has read it.  (The other half
// of S is free as soon as S has been read; half of the next S could be computed
// there meanwhile, which is not done.)  Two row tiles fill a period of 3340
// cycles (a cache: 3900) with 2080 of MMAs.  Measured, calls back to back under
// the power limit: a prompt of 8192 tokens, 32 heads of 128: 568 us, 0.97
// PFLOP/s, 58% of cuBLAS; prompts of 1 to 1800 tokens, 16 heads: 168 us; three
// chunks over a cache 257 us.
//
// Roundings below FP32: P (FP16, as the tensor core's operand: half a step of
// each weight; the sum of weights is taken before it, in FP32) and, for a
// cache, the expanded keys and values: half a step, what they have in FP16
// anyway, the type that they were cached from.  (Keys that are not rounded were
// built in three forms, error 3.4e-4 instead of 7.7e-4 in the norm: two FP16
// parts of each key 376 to 450 us for chunks that take 257; their codes, with
// scales and offsets in the softmax, 303 us, and 351 on fragments of S.)
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "qoq_attn_internal.h"
#include "qoq_attn_device.cuh"
#include "qoq_ptx.cuh"
#include "qoq_quant.cuh"

namespace qoq {
namespace {

// Threads: four softmax warpgroups, for a cache one that loads, and one with the other roles' warps.  (A cache with two
// loaders, keys and values, leaves the softmax 88 registers instead of 96, and one buffer for S: 4% slower.)
__host__ __device__ constexpr int tile_threads(int bits) { return bits ? 768 : 640; }
constexpr int kRows = 256;          // rows of a CTA (two tiles of 128)
constexpr int kKeys = 128;          // keys of a tile
constexpr uint64_t kBudgetNs = 2000000000ull;

__device__ int g_tile_error;        // non-zero after a bounded wait ran out

// One work item: 256 rows of a sequence and KV head, and all or some of their keys.
struct __align__(16) TileItem {
    int row0, rows;         // first row (new token * G + head of the group) in the sequence, rows from there on
    int b, n, hk;           // sequence (-1: the list is at its end), its new tokens, KV head
    int slot;               // where the CTA leaves a partial result: 0 or 1; -1: all keys, the result is final
    int t_seq, first;       // first row of the sequence in the batch, position of its new token 0
    int j0, cnt[2], steps;  // first key tile, key tiles of each row tile, of both
};

constexpr int kChunks = 64;         // chunks of sequences whose first row tiles are kept at hand
constexpr int kAhead = 4;           // items that the scheduler may be ahead
struct TileMisc {
    float row[2][2][128];   // [row tile][half of the columns][row]: what the two threads of a row exchange
    TileItem item[kAhead];
    uint8_t chunk[kChunks]; // chunks, the one with the longest sequence first
    int before[kChunks];    // row tiles (a cache's: key tiles of row tiles and heads) before each of them
    int total;
    uint32_t tmem_slot;
    int abort_flag;
};

template <int D>
struct TileCfg {
    static constexpr int kBlock = kKeys * 128;              // [128 rows][64 channels] FP16, swizzled
    static constexpr int kTile = kBlock * (D / 64);         // K, V or Q of 128 rows
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr int kQ = 0;                            // two Q tiles
    static constexpr int kRing = 2 * kTile;
    static constexpr int kBars = kRing + kSlots * kTile;
    static constexpr int kMisc = kBars + (((2 * kSlots + 9 + 2 * kAhead) * 8 + 15) & ~15);   // barriers, TileMisc
    static constexpr int kSmem = kMisc + sizeof(TileMisc);  // nearly all there is: nothing else is static
    static_assert(kSmem <= 232448, "shared memory of a block");
};

struct TileArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv, ldo;
    uint16_t *out;
    float *part;            // (a cache) [CTAs][2][256][D + 2]: sums of rows, then (maximum, sum of weights) of each
    int4 *joined;           // (a cache) [CTAs]: (sequence or -1, first row, KV head, first CTA) of the row tile whose
                            // keys end in the CTA's share and began in an earlier one's
    AttnCache c;
    AttnBatch a;
    int T, Hq, Hkv, G;
    int few;                // sequences with at most this many rows (n_b * G) are another kernel's
    float scale_log2;       // |scale| * log2(e)
    uint32_t flip;          // 0x80008000 when scale < 0: the sign goes into q
    uint32_t e6, e4;        // 0x64006400, 0x54006400 (expand8, expand4)
    bool wide;              // out's rows begin on 32-byte boundaries: half as many store instructions, which the
                            // load/store unit takes line by line (packed prompts 153 us against 165)
    CUtensorMap map_k, map_v;   // (prompts) [T][Hkv * D], boxes of 64 channels x 128 rows, 128-byte swizzle
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

// 2^x of two numbers on the FMA pipe: 2^x = 2^n 2^f with n = round(x) (adding 1.5 * 2^23 leaves n in the
// low bits), 2^f on [-1/2, 1/2] by the cubic of least relative error, 7.5e-5 (found by linear programming; P is
// rounded to FP16, 4.9e-4, next).  Below 2^-126 the result is some number below 2^-125, from 2^7 on it is
// nothing.
__device__ __forceinline__ void ex2_pair(float &x, float &y)
{
    const uint64_t t = pair(fmaxf(x, -126.0f), fmaxf(y, -126.0f));
    const uint64_t r = add2(t, pair(12582912.0f, 12582912.0f));
    const uint64_t f = add2(t, fma2(r, pair(-1.0f, -1.0f), pair(12582912.0f, 12582912.0f)));
    uint64_t p = fma2(f, pair(0.0551716685f, 0.0551716685f), pair(0.242611125f, 0.242611125f));
    p = fma2(p, f, pair(0.693260968f, 0.693260968f));
    p = fma2(p, f, pair(0.999928057f, 0.999928057f));
    float n0, n1;
    unpair(r, n0, n1);
    unpair(p, x, y);
    x = __uint_as_float(__float_as_uint(x) + (__float_as_uint(n0) << 23));
    y = __uint_as_float(__float_as_uint(y) + (__float_as_uint(n1) << 23));
}

// Pairs of every 8 whose exponential runs on the FMA pipe: the other pipe makes four a clock and SM quarter, which
// alone would take as long as the tensor cores take for the tile.  (The long prompt: 507 us with three, 566 with none.
// A cache's loaders need that pipe themselves: 236 us with none, 241 with two.)
constexpr int kPoly = 3;

// How far below the true maximum the one in use is set, in log2 units: weights count in P down to 2^-25 of one, so down to
// 2^-33 of the largest (a context of 2^17 tokens can hold 2^-16 of its mass below that; at 2^-25, 2^-8), and with full
// FP16 precision down to 2^-22.  64 weights of the largest's size sum to 2^14 then, a quarter of what they may.
constexpr float kBelow = 8.0f;

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

// Registers per thread of the roles; a block of 640 threads is launched with 96 of them for each, one of 768 with 80.
template <int BITS>
struct Regs {
    static constexpr int kSoftmax = BITS ? 96 : 104, kLoader = BITS ? 48 : 0, kRest = BITS ? 48 : 64;
    static_assert(512 * kSoftmax + (BITS ? 128 * kLoader : 0) + 128 * kRest <= tile_threads(BITS) * (BITS ? 80 : 96), "register split");
};

// BITS 0: FP16 rows of the batch itself (prompts); 4 or 8: the cache.
template <int D, int BITS>
__global__ void __launch_bounds__(tile_threads(BITS), 1) attn_tile_kernel(const __grid_constant__ TileArgs p)
{
    using C = TileCfg<D>;
    constexpr int kMmaWarp = BITS ? 20 : 17, kQWarp = kMmaWarp + 1, kQWarps = BITS ? 2 : 1;
    constexpr int kPlanWarp = kQWarp + kQWarps, kReaders = 16 + 1 + kQWarps + (BITS ? 4 : 1);   // warps that read items
    extern __shared__ __align__(1024) uint8_t smem[];
    TileMisc &misc = *reinterpret_cast<TileMisc *>(smem + C::kMisc);
    int &abort_flag = misc.abort_flag;
    float (&s_row)[2][2][128] = misc.row;
    // (the same for a warp's lanes, and the compiler is to know it)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t sbase = smem_addr(smem);
    const uint32_t bars = sbase + C::kBars;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (C::kSlots + s); };
    auto sfull = [&](int t) { return bars + 8u * (2 * C::kSlots + t); };
    auto pfull = [&](int t) { return bars + 8u * (2 * C::kSlots + 2 + t); };
    auto ofull = [&](int t) { return bars + 8u * (2 * C::kSlots + 4 + t); };
    const uint32_t qfull = bars + 8u * (2 * C::kSlots + 6), qempty = qfull + 8, done = qfull + 16;
    auto ifull = [&](int i) { return done + 8 + 8u * i; };
    auto iempty = [&](int i) { return done + 8 + 8u * (kAhead + i); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(full(s), BITS ? 4 : 1);
            mbar_init(empty(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(sfull(t), 1);
            mbar_init(pfull(t), 8);
            mbar_init(ofull(t), 1);
        }
        mbar_init(qfull, kQWarps);
        mbar_init(qempty, 1);
        mbar_init(done, 1);
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(ifull(i), 1);
            mbar_init(iempty(i), kReaders);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&misc.tmem_slot), 512);
        tmem_relinquish();
    }
    // A group's wait: one warp polls, the others sleep in a named barrier instead of polling too; it also makes the
    // answer the same for all of them.
    auto group_wait = [&](int id, int count, bool polls, uint32_t bar, uint32_t parity) -> bool {
        const bool failed = polls && !wait_short(bar, parity, &abort_flag, kBudgetNs);
        return !named_barrier_any(id, count, failed);
    };
    // ---- the items: row tiles of all sequences x KV heads, those that see most first ----
    // row tiles of sequence b (none if it is another kernel's, or has rows outside the batch)
    const int per_chunk = (p.a.B + kChunks - 1) / kChunks;
    auto tiles_of = [&](int b, int &n) -> int {
        const int t0 = __ldg(p.a.cu + b), t1 = __ldg(p.a.cu + b + 1);
        n = t0 >= 0 && t1 <= p.T ? max(0, t1 - t0) : 0;
        const int64_t r = (int64_t)n * p.G;
        return r > p.few ? (int)((r + kRows - 1) / kRows) : 0;
    };
    // (a cache) key tiles that row tile `row0` of a sequence sees, at least one: even a row tile that sees nothing is
    // worked on
    auto units_of = [&](int first, int n, int row0) -> int {
        const int r = min(n * p.G - row0, kRows) - 1;
        const int keys = min(first + (row0 + r) / p.G + 1, p.a.table_pages * p.a.page_size);
        return max(1, (keys + kKeys - 1) / kKeys);
    };
    auto first_of = [&](int b, int n) -> int { return max(0, __ldg(p.a.kv_len + b)) - n; };
    if (warp < kChunks / 32) {
        int *length = reinterpret_cast<int *>(misc.row);
        int sum = 0, n, len = 0;
        for (int b = threadIdx.x * per_chunk; b < min(p.a.B, ((int)threadIdx.x + 1) * per_chunk); ++b) {
            const int tiles = tiles_of(b, n);
            len = max(len, BITS ? __ldg(p.a.kv_len + b) : n);
            if (BITS) {
                const int first = first_of(b, n);
                for (int i = 0; i < tiles; ++i) sum += units_of(first, n, i * kRows) * p.Hkv;
            } else {
                sum += tiles;
            }
        }
        length[threadIdx.x] = sum > 0 ? len : -1;
        named_barrier(1, kChunks);
        int rank = 0;                                // chunks by their longest sequence
        for (int j = 0; j < kChunks; ++j) {
            const int x = length[j], y = length[threadIdx.x];
            rank += x > y || (x == y && j < (int)threadIdx.x);
        }
        misc.chunk[rank] = threadIdx.x;
        misc.before[rank] = sum;
    }
    __syncthreads();
    if (warp == 0) {
        const int x = misc.before[2 * lane], y = misc.before[2 * lane + 1];
        int z = x + y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += u;
        }
        misc.before[2 * lane] = z - x - y;
        misc.before[2 * lane + 1] = z - y;
        if (lane == 31) misc.total = z;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc.tmem_slot;
    // The next item, from the scheduler's ring; false at the end of the list, or when a wait ran out.  Every role walks
    // the same list.  Warps that meet in barriers take an item together or not at all: get_together().
    int turn = 0;                                    // items read so far
    TileItem w;
    auto take = [&](bool there) -> bool {
        if (!there) return false;
        const int i = turn % kAhead;
        w = misc.item[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty(i));
        ++turn;
        return w.b >= 0;
    };
    auto get = [&]() -> bool {
        return take(__all_sync(0xffffffffu, wait_short(ifull(turn % kAhead), (uint32_t)(turn / kAhead) & 1, &abort_flag, kBudgetNs)));
    };
    auto get_together = [&](int id, int count, bool polls) -> bool {
        return take(group_wait(id, count, polls, ifull(turn % kAhead), (uint32_t)(turn / kAhead) & 1));
    };

    if (BITS ? warp >= 20 : warp >= 16) {
        // ------------------------------------- MMA (and the prompts' loader) --
        regs_down<Regs<BITS>::kRest>();
        if (warp == kMmaWarp) {
            const uint32_t lead = elect_lane();
            auto uniform = [](bool x) { return (bool)__all_sync(0xffffffffu, x); };
            const uint32_t is = idesc_f16_m128(kKeys, false), io = idesc_f16_m128(D, true);
            const uint32_t q_lo = desc_sw128_lo(sbase + C::kQ, 1), k_lo = desc_sw128_lo(sbase + C::kRing, 1);
            const uint32_t v_lo = desc_sw128_lo(sbase + C::kRing, C::kBlock >> 4);
            auto scores = [&](int t, int slot) {
                const uint32_t qa = q_lo + t * (C::kTile >> 4), kb = k_lo + slot * (C::kTile >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * (C::kBlock >> 4) + 2 * (kk & 3);
                    mma_f16_ss(lead, tmem + 128 * t, qa + off, kb + off, kDescSw128Hi, kDescSw128Hi, is, kk > 0);
                }
                mma_commit_lead(lead, sfull(t));
            };
            auto values = [&](int t, int slot, bool accumulate) {
                const uint32_t vb = v_lo + slot * (C::kTile >> 4);
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    mma_f16_ts(lead, tmem + 256 + D * t, tmem + 128 * t + 8 * kk, vb + 128 * kk, kDescSw128Hi, io,
                               accumulate || kk > 0);
            };
            // The ring's units go K V K V ... through all items: K of an item's step i is unit base + 2i, V the next.
            int base = 0, slot_k = 0, done_q = 0, done_p[2] = {0, 0};        // units, their slot, uses of qfull and pfull
            bool ok = true;
            auto ready = [&](int unit, int slot) {
                return uniform(wait_short(full(slot), (uint32_t)(unit / C::kSlots) & 1, &abort_flag, kBudgetNs));
            };
            auto next = [](int slot) { return slot + 1 == C::kSlots ? 0 : slot + 1; };
            while (ok && get()) {
                if (w.steps == 0) continue;
                ok = uniform(wait_short(qfull, (uint32_t)done_q++ & 1, &abort_flag, kBudgetNs)) && ready(base, slot_k);
                if (!ok) break;
                tc_fence_after();
                // (S goes over P of the last item: MMAs run in the order they were issued)
                for (int t = 0; t < 2; ++t)
                    if (w.cnt[t] > 0) scores(t, slot_k);
                mma_commit_lead(lead, empty(slot_k));
                if (w.steps == 1) mma_commit_lead(lead, qempty);
                for (int i = 0; i < w.steps && ok; ++i) {
                    const int slot_v = next(slot_k);
                    slot_k = next(slot_v);
                    bool have_k = false;
                    ok = ready(base + 2 * i + 1, slot_v);
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (i >= w.cnt[t]) continue;
                        ok = uniform(wait_short(pfull(t), (uint32_t)done_p[t]++ & 1, &abort_flag, kBudgetNs));
                        if (!ok) break;
                        tc_fence_after();
                        values(t, slot_v, i > 0);
                        if (i + 1 < w.cnt[t]) {
                            if (!have_k) {
                                ok = have_k = ready(base + 2 * i + 2, slot_k);
                                if (!ok) break;
                                tc_fence_after();
                            }
                            scores(t, slot_k);
                        } else {
                            mma_commit_lead(lead, ofull(t));
                        }
                    }
                    if (!ok) break;
                    mma_commit_lead(lead, empty(slot_v));
                    if (i + 1 < w.steps) mma_commit_lead(lead, empty(slot_k));
                    if (i + 2 == w.steps) mma_commit_lead(lead, qempty);     // the item's last S was just issued
                }
                base += 2 * w.steps;
            }
            // However the list ended, what was issued finishes before tensor memory and the barriers go.
            mma_commit_lead(lead, done);
            const uint64_t end = global_timer_ns() + 200000000ull;
            while (!mbar_try_wait(done, 0) && global_timer_ns() < end) {
            }
        }
        if (warp >= kQWarp && warp < kQWarp + kQWarps) {
            // Q of the next item as soon as the last S of this one is done: 256 rows, zeros past the end
            // Four lanes to a row, its vectors v0, v0 + 4, ...; a lane's rows are a multiple of 8 apart, so that one
            // swizzle serves them.
            constexpr int kPass = 8 * kQWarps, kN = D / 32;
            const int r0 = 8 * (warp - kQWarp) + lane / 4, v0 = lane % 4;
            const int dt = kPass / p.G, dg = kPass % p.G;    // a pass further: tokens, heads
            uint32_t at[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) at[j] = sbase + C::kQ + ((v0 + 4 * j) >> 3) * C::kBlock + swz(r0, v0 + 4 * j);
            int used = 0;
            while (get()) {
                if (w.steps == 0) continue;
                if (used > 0 && !__all_sync(0xffffffffu, wait_short(qempty, (uint32_t)(used - 1) & 1, &abort_flag, kBudgetNs))) break;
                ++used;
                int g = (w.row0 + r0) % p.G;
                const uint16_t *src = p.q + (int64_t)(w.t_seq + (w.row0 + r0) / p.G) * p.ldq + (size_t)w.hk * p.G * D + 8 * v0;
                auto offset = [](int r) { return (r >> 7) * C::kTile + (r & 127) * 128; };
#pragma unroll 2
                for (int r = r0; r < kRows; r += kPass) {
                    const uint32_t off = offset(r - r0 % 8) - offset(r0 - r0 % 8);
                    const bool in = r < w.rows;
#pragma unroll
                    for (int j = 0; j < kN; ++j) cp_async16(at[j] + off, in ? src + g * D + 32 * j : p.q, in);
                    src += dt * p.ldq;
                    g += dg;
                    if (g >= p.G) {
                        g -= p.G;
                        src += p.ldq;
                    }
                }
                cp_async_commit();
                cp_async_wait<0>();
                if (p.flip) {                                // each lane its own vectors
#pragma unroll 2
                    for (int r = r0; r < kRows; r += kPass) {
                        const uint32_t off = offset(r - r0 % 8) - offset(r0 - r0 % 8);
#pragma unroll
                        for (int j = 0; j < kN; ++j) {
                            const uint4 x = ld_shared16(at[j] + off);
                            st_shared16(at[j] + off, make_uint4(x.x ^ p.flip, x.y ^ p.flip, x.z ^ p.flip, x.w ^ p.flip));
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull);
            }
            cp_async_wait<0>();
        }
        if (warp == kPlanWarp) {
            // the chunk of sequences that begins at or before place x of the list, with x counted from its beginning
            auto chunk_at = [&](int &x) -> int {
                int lo = 0, hi = kChunks - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (misc.before[mid] <= x) lo = mid;
                    else hi = mid - 1;
                }
                x -= misc.before[lo];
                return lo;
            };
            int emitted = 0;
            // hands w over, with key tiles [j0, j1) of its rows; false when a wait ran out
            auto emit = [&](int j1) -> bool {
                if (w.b >= 0) {
                    w.rows = w.n * p.G - w.row0;
                    w.t_seq = __ldg(p.a.cu + w.b);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int r = min(w.rows, 128 * (t + 1)) - 1;
                        int last = w.rows > 128 * t ? max(0, w.first + (w.row0 + r) / p.G + 1) : 0;   // keys its last row sees
                        if (BITS) last = min(last, p.a.table_pages * p.a.page_size);
                        w.cnt[t] = max(0, min((last + kKeys - 1) / kKeys, j1) - w.j0);
                    }
                    w.steps = max(w.cnt[0], w.cnt[1]);
                }
                const int i = emitted % kAhead;
                if (emitted >= kAhead &&
                    !__all_sync(0xffffffffu, wait_short(iempty(i), (uint32_t)(emitted / kAhead - 1) & 1, &abort_flag, kBudgetNs)))
                    return false;
                if (lane == 0) {
                    misc.item[i] = w;
                    mbar_arrive(ifull(i));
                }
                ++emitted;
                return true;
            };
            bool ok = true;
            if (BITS == 0) {
                // whole row tiles, in rounds that go to and fro over the CTAs, since they get smaller
                const int items = misc.total * p.Hkv;
                for (int k = 0; ok; ++k) {
                    const int x = k * (int)gridDim.x + (k & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
                    if (x >= items) break;
                    w.hk = x % p.Hkv;
                    w.slot = -1;
                    w.j0 = w.first = 0;
                    int tile = x / p.Hkv, count;
                    for (w.b = misc.chunk[chunk_at(tile)] * per_chunk; w.b < p.a.B; ++w.b) {
                        count = tiles_of(w.b, w.n);
                        if (tile < count) break;
                        tile -= count;
                    }
                    if (w.b >= p.a.B) break;                 // (the sums ran over: rows counted in several sequences)
                    w.row0 = (count - 1 - tile) * kRows;
                    ok = emit(1 << 30);
                }
            } else {
                // An equal share of all key tiles: CTA c of P takes units c S / P .. (c + 1) S / P - 1 of the list of
                // (row tile, head, key tile).  A row tile whose keys are shared out leaves a part in each CTA.
                const int ctas = min((int)gridDim.x, misc.total), c = blockIdx.x;
                if (lane == 0) p.joined[c] = make_int4(-1, 0, 0, 0);
                int at = c < ctas ? (int)((int64_t)misc.total * c / ctas) : 0;
                const int end = c < ctas ? (int)((int64_t)misc.total * (c + 1) / ctas) : 0;
                if (at < end) {
                    int x = at, lo = chunk_at(x), units = 0;
                    int in_chunk = 0;
                    // the first row tile: x becomes the place in it
                    bool found = false;
                    while (!found) {
                        w.b = misc.chunk[lo] * per_chunk + in_chunk;
                        if (w.b >= p.a.B) break;             // (the sums ran over: rows counted in several sequences)
                        const int tiles = tiles_of(w.b, w.n);
                        w.first = first_of(w.b, w.n);
                        for (w.row0 = (tiles - 1) * kRows; w.row0 >= 0; w.row0 -= kRows) {
                            units = units_of(w.first, w.n, w.row0);
                            found = x < units * p.Hkv;
                            if (found) break;
                            x -= units * p.Hkv;
                        }
                        if (!found) ++in_chunk;
                    }
                    w.hk = found ? x / units : 0;
                    w.j0 = found ? x % units : 0;
                    while (ok && found) {
                        const int j1 = min(units, w.j0 + end - at);
                        w.slot = w.j0 == 0 && j1 == units ? -1 : w.j0 == 0 ? 1 : 0;
                        if (w.slot == 0 && j1 == units && lane == 0)
                            p.joined[c] = make_int4(w.b, w.row0, w.hk,
                                                    (int)(((int64_t)(at - w.j0 + 1) * ctas - 1) / misc.total));
                        ok = emit(j1);
                        at += j1 - w.j0;
                        if (at >= end) break;
                        w.j0 = 0;
                        if (++w.hk < p.Hkv) continue;
                        w.hk = 0;
                        w.row0 -= kRows;
                        while (w.row0 < 0) {                 // the next sequence with tiles
                            if (++in_chunk == per_chunk || misc.chunk[lo] * per_chunk + in_chunk >= p.a.B) {
                                in_chunk = 0;
                                found = ++lo < kChunks;
                                if (!found) break;
                            }
                            w.b = misc.chunk[lo] * per_chunk + in_chunk;
                            w.row0 = w.b < p.a.B ? (tiles_of(w.b, w.n) - 1) * kRows : -1;
                            w.first = w.b < p.a.B ? first_of(w.b, w.n) : 0;
                        }
                        if (found) units = units_of(w.first, w.n, w.row0);
                    }
                }
            }
            w.b = -1;
            if (ok) emit(0);
        }
        if (BITS == 0 && warp == 16) {
            // TMA, except for the last values of a sequence: rows behind it are another's, or nobody's, and may hold
            // anything, and a weight of zero does not silence an infinity.  (Keys there only make scores that are
            // masked.)
            int unit = 0;
            bool ok = true;
            while (ok && get()) {
                const bool ragged = w.steps > 0 && (w.j0 + w.steps) * kKeys > w.n;
                for (int i = 0; i < 2 * w.steps; ++i, ++unit) {
                    const int slot = unit % C::kSlots;
                    ok = unit < C::kSlots ||
                         __all_sync(0xffffffffu, wait_short(empty(slot), (uint32_t)(unit / C::kSlots - 1) & 1, &abort_flag, kBudgetNs));
                    if (!ok) break;
                    const uint32_t dst = sbase + C::kRing + slot * C::kTile;
                    const int key0 = (w.j0 + (i >> 1)) * kKeys;
                    if (ragged && i == 2 * w.steps - 1) {
                        constexpr int kVecs = D / 8;
                        for (int e = lane; e < kKeys * kVecs; e += 32) {
                            const int row = e / kVecs, vec = e % kVecs;
                            const bool in = key0 + row < w.n;
                            cp_async16(dst + (vec >> 3) * C::kBlock + swz(row, vec),
                                       in ? p.v + (int64_t)(w.t_seq + key0 + row) * p.ldv + (size_t)w.hk * D + vec * 8 : p.v, in);
                        }
                        cp_async_commit();
                        cp_async_wait<0>();
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full(slot));
                    } else if (lane == 0) {
                        mbar_arrive_expect_tx(full(slot), C::kTile);
#pragma unroll
                        for (int blk = 0; blk < D / 64; ++blk)
                            tma_load_2d(dst + blk * C::kBlock, i & 1 ? &p.map_v : &p.map_k, w.hk * D + 64 * blk,
                                        w.t_seq + key0, full(slot));
                    }
                }
            }
            if (lane == 0) {            // however the list ended, copies in flight land before the shared memory goes
                const uint64_t end = global_timer_ns() + 200000000ull;
                for (int u = max(0, unit - C::kSlots); u < unit; ++u)
                    while (!mbar_try_wait(full(u % C::kSlots), (uint32_t)(u / C::kSlots) & 1) && global_timer_ns() < end) {
                    }
            }
        }
    } else if (BITS && warp >= 16) {
        // ------------------------------------------------ loaders of a cache --
        regs_down<Regs<BITS ? BITS : 4>::kLoader>();
        {
            // One warpgroup brings the keys and the values in turn.  kLanes lanes share a row's bytes, 16 each; a thread's
            // kLanes rows lie in one granule of 16 tokens, kGap apart, so one page and constant offsets serve them.
            constexpr int kB = BITS ? BITS : 4;
            constexpr int kRowBytes = D * kB / 8, kLanes = kRowBytes / 16, kGap = 16 / kLanes;
            constexpr int kVecs = 128 / kB / 8;                      // 16-byte vectors of 8 channels from 16 bytes of codes
            const int tid = threadIdx.x & 127, part = tid % kLanes;
            const int r0 = 16 * (tid / 16) + tid % 16 / kLanes;      // r0 % 8 is below kGap, and the other rows' r % 8 are
                                                                     // r0 % 8 ^ (kGap i % 8)
            constexpr int kBatch = kLanes < 4 ? kLanes : 4, kBatches = kLanes / kBatch;    // rows in registers at a time
            uint4 c[kBatch];
            uint32_t pr[kBatch];
            int page = -1;                                           // of the next step to be fetched
            auto look_up = [&](int step) {
                const int pos = (w.j0 + step) * kKeys + r0;
                page = (pos & ~15) < w.first + w.n ? page_of(p.a, w.b, pos) : -1;
            };
            auto fetch = [&](int u, int batch) {                     // u: keys (even) and values (odd) of the steps
                const int step = u >> 1;
                const int pos = (w.j0 + step) * kKeys + r0 + batch * kBatch * kGap, end = w.first + w.n;
                // (a pool of 2^32 rows would not fit the GPU)
                const uint32_t row = ((uint32_t)page * p.Hkv + w.hk) * p.a.page_size + (pos & (p.a.page_size - 1));
                const uint8_t *src = (u & 1 ? p.c.v_codes : p.c.k_codes) + part * 16 + (size_t)row * kRowBytes;
                const uint32_t *par = reinterpret_cast<const uint32_t *>(u & 1 ? p.c.v_par : p.c.k_par) + row;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    c[i] = make_uint4(0, 0, 0, 0);
                    pr[i] = 0;
                    if (page >= 0 && pos + kGap * i < end) {         // what nobody sees becomes zeros
                        c[i] = __ldg(reinterpret_cast<const uint4 *>(src + kGap * i * kRowBytes));
                        pr[i] = __ldg(par + kGap * i);
                    }
                }
                if ((u & 1) && batch == kBatches - 1) look_up(step + 1);
            };
            // Vector v of the thread's codes is vector kVecs * part + v of the row.  Lanes of the row's upper half store
            // theirs in another order, so that eight lanes meet eight bank groups.
            const int twist = D == 128 && part >= kLanes / 2 ? kVecs / 2 : 0;
            uint32_t at[kVecs];
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                const int vec = kVecs * part + (u ^ twist);
                at[u] = (uint32_t)((vec >> 3) * C::kBlock) + swz(r0, vec);
            }
            auto expand = [&](int slot, int batch) {
                const uint32_t dst = sbase + C::kRing + slot * C::kTile + batch * kBatch * kGap * 128;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const uint32_t cw[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
                    for (int u = 0; u < kVecs; ++u) {
                        constexpr int kHalf = kVecs / 2;
                        uint4 x;
                        if (kB == 4) x = expand4(twist ? cw[u ^ kHalf] : cw[u], pr[i], p.e4);
                        else x = expand8(twist ? cw[2 * (u ^ kHalf) % 4] : cw[2 * u % 4],
                                         twist ? cw[(2 * (u ^ kHalf) + 1) % 4] : cw[(2 * u + 1) % 4], pr[i], p.e6);
                        // (a batch's rows are a multiple of 8 from the first batch's: the same swizzle)
                        st_shared16(dst + (at[u] ^ ((kGap * i & 7) << 4)) + kGap * i * 128, x);
                    }
                }
            };
            static_assert(kBatches == 1 || kBatch * kGap % 8 == 0, "swizzle of the batches");
            int unit = 0;
            bool ok = true;
            while (ok && get_together(6, 128, (warp & 3) == 0)) {
                if (w.steps == 0) continue;
                look_up(0);
                fetch(0, 0);
                for (int i = 0; i < 2 * w.steps; ++i, ++unit) {
                    const int slot = unit % C::kSlots;
                    ok = unit < C::kSlots ||
                         group_wait(6, 128, (warp & 3) == 0, empty(slot), (uint32_t)(unit / C::kSlots - 1) & 1);
                    if (!ok) break;
#pragma unroll
                    for (int x = 0; x < kBatches; ++x) {
                        expand(slot, x);
                        if (x + 1 < kBatches) fetch(i, x + 1);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full(slot));
                    if (i + 1 < 2 * w.steps) fetch(i + 1, 0);
                }
            }
        }
    } else {
        // -------------------------------------------------------- softmax --
        regs_up<Regs<BITS>::kSoftmax>();
        // row tile, half of its columns, row of the tile (= lane of tensor memory)
        const int t = warp >> 3, h = warp >> 2 & 1, r = (warp & 3) * 32 + lane;
        constexpr int kCols = kKeys / 2, kOut = D / 2;               // of S and of O that are this thread's
        const int row = 128 * t + r;                                 // of the item
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = tmem + 128 * t + kCols * h + lanes;      // S; P goes over the tile's first 64 columns
        const uint32_t tp = tmem + 128 * t + kCols / 2 * h + lanes;
        const uint32_t to = tmem + 256 + D * t + kOut * h + lanes;
        const float sl = p.scale_log2;
        const int mates = 8 + 4 * t + (warp & 3);                    // barrier of the two warps that share 32 rows
        int used = 0, finished = 0;                                  // uses of sfull, of ofull
        bool ok = true;
        while (ok && get_together(2 + t, 256, (warp & 7) == 0)) {
        const bool real = row < w.rows;
        const int tok = real ? (w.row0 + row) / p.G : 0;
        const int see = real ? w.first + tok + 1 : 0;                // keys 0 .. see - 1 are seen
        const int see_min = __reduce_min_sync(0xffffffffu, real ? see : INT_MAX);   // (what other rows come to is not used)
        float m = -INFINITY, l = 0.0f;                               // maximum in use (log2 units), sum of the columns
        // (a cache) the table's entry for a 16-token piece of step i's columns, a lane each; fetched a step ahead
        auto piece = [&](int i) {
            const int place = ((w.j0 + i) * kKeys + kCols * h + 16 * lane) >> p.a.page_shift;
            return BITS && lane < 4 && place < p.a.table_pages ? __ldg(p.a.table + (size_t)w.b * p.a.table_pages + place) : -1;
        };
        int page = piece(0);
        for (int i = 0; i < w.cnt[t]; ++i) {
            const int key0 = (w.j0 + i) * kKeys + kCols * h;
            // (cache) which 16-token pieces of the columns are there
            uint32_t there = 0xFu;
            if (BITS) {
                there = __ballot_sync(0xffffffffu, page >= 0 && page < p.a.pages);
                page = piece(i + 1);
            }
            ok = group_wait(2 + t, 256, (warp & 7) == 0, sfull(t), (uint32_t)used++ & 1);
            if (!ok) break;
            tc_fence_after();
            const int lim = see - key0;
            const bool masked = see_min < key0 + kCols || there != 0xFu;
            // -inf over the columns [c0, c0 + 16) that the row does not see
            auto mask = [&](uint32_t (&x)[16], int c0) {
                const int left = (there >> (c0 / 16)) & 1 ? lim - c0 : 0;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (c >= left) x[c] = 0xFF800000u;
            };
            // P = 2^(s - m), FP16, with the maximum in use, 16 columns at a time, the next 16 on their way from tensor
            // memory.  The maximum may lag behind: as long as a thread's weights sum to what FP16 holds, each of them
            // fits, and no maximum has to be taken.  Otherwise, and for the first keys that a row sees, the two warps of
            // the rows take it (less kBelow), rescale what they have and weigh the tile again.
            uint32_t pk[kCols / 2];
            for (int round = 0;; ++round) {
                if (round > 0 || i > 0) {                            // (an item's first keys have no maximum to use)
                    const float sub = m == -INFINITY ? 0.0f : -m;
                    const uint64_t sl2 = pair(sl, sl), sub2 = pair(sub, sub);
                    uint64_t sum2[2] = {0, 0};
                    float high = -INFINITY;
                    uint32_t x[2][16];
                    tmem_ld16_async(ts, x[0]);
#pragma unroll
                    for (int c0 = 0; c0 < kCols; c0 += 16) {
                        uint32_t (&y)[16] = x[c0 / 16 % 2];
                        tmem_wait_ld16(y);
                        if (c0 + 16 < kCols) tmem_ld16_async(ts + c0 + 16, x[(c0 / 16 + 1) % 2]);
                        if (masked) mask(y, c0);
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            float e0, e1;
                            unpair(fma2(pair(__uint_as_float(y[2 * u]), __uint_as_float(y[2 * u + 1])), sl2, sub2), e0, e1);
                            if (BITS == 0 && u < kPoly) {
                                high = max_nan(max_nan(high, e0), e1);   // (a sum would not show what is out of its range, or NaN)
                                ex2_pair(e0, e1);
                            } else {
                                e0 = ex2(e0);
                                e1 = ex2(e1);
                            }
                            sum2[u & 1] = add2(sum2[u & 1], pair(e0, e1));
                            const __half2 x2 = __floats2half2_rn(e0, e1);
                            pk[c0 / 2 + u] = *reinterpret_cast<const uint32_t *>(&x2);
                        }
                    }
                    float s0, s1;
                    unpair(add2(sum2[0], sum2[1]), s0, s1);
                    s0 += s1;
                    // (also: everyone has read S before anyone writes P over it)
                    const bool again = named_barrier_any(mates, 64, round == 0 && (s0 > 65504.0f || high > 15.0f || (m == -INFINITY && lim > 0 && s0 == s0)));
                    if (!again) {
                        l += BITS || high == high ? s0 : high;
                        break;
                    }
                }
                float top = -INFINITY;
#pragma unroll 1
                for (int c0 = 0; c0 < kCols; c0 += 16) {
                    uint32_t y[16];
                    tmem_ld16(ts + c0, y);
                    mask(y, c0);
#pragma unroll
                    for (int c = 0; c < 16; ++c) top = fmaxf(top, __uint_as_float(y[c]));
                }
                s_row[t][h][r] = top * sl;
                named_barrier(mates, 64);
                const float m1 = fmaxf(m, fmaxf(s_row[t][0][r], s_row[t][1][r]) - kBelow);
                const float keep = m == -INFINITY ? 0.0f : ex2(m - m1);
                m = m1;
                l *= keep;
                // S of this step is complete, so is P V of the last one (issued before it)
#pragma unroll 1
                for (int c = 0; c < (i > 0 ? kOut : 0); c += 16) {
                    uint32_t o[16];
                    tmem_ld16(to + c, o);
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * keep);
                    tmem_st16(to + c, o);
                }
                named_barrier(mates, 64);       // s_row has been read
            }
            tmem_st32(tp, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull(t));
        }
        if (!ok) break;
        // ---- O out ----
        if (w.cnt[t] > 0) {
            ok = group_wait(2 + t, 256, (warp & 7) == 0, ofull(t), (uint32_t)finished++ & 1);
            if (!ok) break;
            tc_fence_after();
        }
        {
            s_row[t][h][r] = l;
            named_barrier(mates, 64);
            l = s_row[t][0][r] + s_row[t][1][r];
            named_barrier(mates, 64);       // s_row has been read: the next item, without keys for this row tile, writes it at once
            const int g = real ? (w.row0 + row) % p.G : 0;
            if (BITS == 0 || w.slot < 0) {
                const bool none = BITS && l == 0.0f;                 // the row saw nothing (a sum that is NaN is not hidden)
                const float inv = none ? 0.0f : 1.0f / l;
                uint16_t *dst = p.out + (int64_t)(w.t_seq + tok) * p.ldo + (size_t)(w.hk * p.G + g) * D + kOut * h;
#pragma unroll
                for (int c = 0; c < kOut; c += 16) {
                    uint32_t o[16], y[8];
                    if (w.cnt[t] > 0) tmem_ld16(to + c, o);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const __half2 x = __floats2half2_rn(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv);
                        y[u] = none ? 0u : *reinterpret_cast<const uint32_t *>(&x);
                    }
                    const uint4 a = make_uint4(y[0], y[1], y[2], y[3]), b = make_uint4(y[4], y[5], y[6], y[7]);
                    if (real) {
                        if (p.wide) {
                            st_global32(dst + c, a, b);
                        } else {
                            reinterpret_cast<uint4 *>(dst + c)[0] = a;
                            reinterpret_cast<uint4 *>(dst + c)[1] = b;
                        }
                    }
                }
            } else {
                float *mine = p.part + ((size_t)blockIdx.x * 2 + w.slot) * kRows * (D + 2);
                float4 *dst = reinterpret_cast<float4 *>(mine) + kOut / 4 * h * kRows + row;
                if (h == 0) reinterpret_cast<float2 *>(mine + kRows * D)[row] = make_float2(m, l);
#pragma unroll
                for (int c = 0; c < (w.cnt[t] > 0 ? kOut : 0); c += 16) {
                    uint32_t o[16];
                    tmem_ld16(to + c, o);
                    if (real && l > 0.0f) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            reinterpret_cast<uint4 *>(dst)[(c / 4 + u) * kRows] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
                        }
                    }
                }
            }
        }
        // (O has been read: the next item's first P V, which writes it, waits for this thread's next P)
        tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (BITS) {
        grid_launch_dependents();
        // This grid may run beside the one before it, and does not need its results; but whoever waits for this one
        // waits for both.
        grid_dependency_wait();
    }
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && abort_flag) atomicExch(&g_tile_error, 1);
}

// Joins a cache's row tiles that several CTAs share: CTA (x, y) the one that ended in CTA x's share, eight rows of it,
// four channels per thread; the parts in order.  A part holds four channels of all rows, then the next four: what the
// warps that write it (a row per thread) and those that read it here take in whole lines.
constexpr int kJoinRows = 8;

template <int D>
__global__ void __launch_bounds__(kJoinRows *D / 4) attn_tile_join_kernel(const float *__restrict__ part,
                                                                          const int4 *__restrict__ joined, AttnBatch a,
                                                                          int Hkv, int G, uint16_t *__restrict__ out, int64_t ldo)
{
    grid_dependency_wait();
    const int last = blockIdx.x, row = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, at = threadIdx.x / kJoinRows;
    const int4 j = joined[last];
    if (j.x < 0) return;
    const int t0 = __ldg(a.cu + j.x), n = __ldg(a.cu + j.x + 1) - t0;
    if (row >= n * G - j.y) return;
    float M = -INFINITY, L = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kAhead = 4;                        // parts loaded at a time
    for (int c0 = j.w; c0 <= last; c0 += kAhead) {
        float2 ml[kAhead];
        float4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int c = c0 + u;
            ml[u] = make_float2(0.0f, 0.0f);
            if (c <= last) {
                const float *src = part + ((size_t)c * 2 + (c == j.w ? 1 : 0)) * kRows * (D + 2);
                ml[u] = reinterpret_cast<const float2 *>(src + kRows * D)[row];
                x[u] = reinterpret_cast<const float4 *>(src)[at * kRows + row];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (ml[u].y == 0.0f) continue;           // saw nothing, and wrote no sums
            const float m1 = fmaxf(M, ml[u].x), f0 = M == -INFINITY ? 0.0f : ex2(M - m1), f1 = ex2(ml[u].x - m1);
            M = m1;
            L = fmaf(L, f0, ml[u].y * f1);
            v = make_float4(fmaf(v.x, f0, x[u].x * f1), fmaf(v.y, f0, x[u].y * f1), fmaf(v.z, f0, x[u].z * f1),
                            fmaf(v.w, f0, x[u].w * f1));
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int r = j.y + row;
    uint16_t *dst = out + (int64_t)(t0 + r / G) * ldo + (size_t)(j.z * G + r % G) * D + 4 * at;
    const __half2 y0 = __floats2half2_rn(v.x * inv, v.y * inv), y1 = __floats2half2_rn(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&y0), *reinterpret_cast<const uint32_t *>(&y1));
}

constexpr int kMaxTileCtas = 160;       // sizes the workspace

template <int D, int BITS>
cudaError_t launch_tile(const TileArgs &p, cudaStream_t stream, bool early, bool join)
{
    // one CTA per SM (shared and tensor memory allow no more), each with its share of the work
    const int64_t items = BITS ? row_tiles(p.T, p.a.B, p.G, p.few) * p.Hkv * 64 : row_tiles(p.T, p.a.B, p.G, p.few) * p.Hkv;
    const int ctas = (int)std::min<int64_t>(items, std::min(attn_sms(), kMaxTileCtas));
    if (join)
        return launch_kernel(attn_tile_join_kernel<D>, dim3(ctas, kRows / kJoinRows), kJoinRows * D / 4, 0, stream, true,
                             (const float *)p.part, (const int4 *)p.joined, p.a, p.Hkv, p.G, p.out, p.ldo);
    auto kernel = attn_tile_kernel<D, BITS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3(ctas), tile_threads(BITS), TileCfg<D>::kSmem, stream, early, p);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

cudaError_t encode_rows(CUtensorMap *map, const uint16_t *x, int T, int width, int64_t ld)
{
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dim[2] = {(cuuint64_t)width, (cuuint64_t)T}, stride[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, kKeys}, one[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<uint16_t *>(x), dim, stride, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr float kLog2e = 1.4426950408889634f;

bool wide_rows(const uint16_t *out, int64_t ldo)
{
    return (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && ldo % 16 == 0;
}

void set_scale(TileArgs &p, float scale)
{
    // a zero scale keeps a tiny one: the same uniform weights, and no 0 * infinity at masked scores
    p.scale_log2 = fmaxf(fabsf(scale) * kLog2e, 1e-30f);
    p.flip = scale < 0.0f ? 0x80008000u : 0u;
}

}  // namespace

int64_t row_tiles(int T, int B, int G, int few)
{
    // every sequence that has tiles wastes at most a part of one
    const int64_t rows = (int64_t)T * G, most = few > 0 ? rows / (few + 1) : T;
    return rows / kRows + (B < most ? B : most);
}

cudaError_t launch_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                                    int64_t ldv, int T, int Hq, int Hkv, int d, const AttnBatch &a, float scale,
                                    uint16_t *out, int64_t ldo, cudaStream_t stream)
{
    TileArgs p{q, k, v, ldq, ldk, ldv, ldo, out, nullptr, nullptr, AttnCache{}, a, T, Hq, Hkv, Hq / Hkv, 0, 0.0f, 0u, 0x64006400u, 0x54006400u, wide_rows(out, ldo), {}, {}};
    set_scale(p, scale);
    cudaError_t e = encode_rows(&p.map_k, k, T, Hkv * d, ldk);
    if (e == cudaSuccess) e = encode_rows(&p.map_v, v, T, Hkv * d, ldv);
    if (e != cudaSuccess) return e;
    return d == 128 ? launch_tile<128, 0>(p, stream, false, false) : launch_tile<64, 0>(p, stream, false, false);
}

size_t tiles_workspace(int d)
{
    return (size_t)kMaxTileCtas * (sizeof(int4) + 2 * kRows * (d + 2) * sizeof(float));
}

bool tiles_fit(int64_t tiles, int Hkv, int table_pages, int page_size)
{
    return tiles * Hkv * ((int64_t)table_pages * page_size / kKeys + 2) < ((int64_t)1 << 31);
}

cudaError_t launch_paged_tiles(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d, const AttnCache &c,
                               const AttnBatch &a, int few, float scale, uint16_t *out, int64_t ldo, void *workspace,
                               cudaStream_t stream, bool early, bool join)
{
    int4 *joined = reinterpret_cast<int4 *>(workspace);
    TileArgs p{q, nullptr, nullptr, ldq, 0, 0, ldo, out, reinterpret_cast<float *>(joined + kMaxTileCtas), joined, c, a, T, Hq,
               Hkv, Hq / Hkv, few, 0.0f, 0u, 0x64006400u, 0x54006400u, wide_rows(out, ldo), {}, {}};
    set_scale(p, scale);
    if (d == 128) return c.bits == 4 ? launch_tile<128, 4>(p, stream, early, join) : launch_tile<128, 8>(p, stream, early, join);
    return c.bits == 4 ? launch_tile<64, 4>(p, stream, early, join) : launch_tile<64, 8>(p, stream, early, join);
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
