// Backward pass of the fused attention for sm_103a. With G = Hq / Hkv,
//   P_ij  = exp(scale <q_i, k_j> + mask_ij - lse_i)     (recomputed, never stored)
//   dV_j  = sum_i P_ij dO_i
//   dP_ij = <dO_i, v_j>
//   dS_ij = P_ij (dP_ij - delta_i),   delta_i = <dO_i, O_i>
//   dQ_i  = scale sum_j dS_ij k_j,    dK_j = scale sum_i dS_ij q_i
// where the sums for dK and dV run over the G query heads of a K/V head too.
//
// Two kernels, of which each owns what it writes:
//   bwd_dkv_kernel  a tile is (b, K/V head, 128 keys); it walks the queries that
//                   see the keys, of all G heads, and holds dK and dV in TMEM;
//   bwd_dq_kernel   a tile is (b, query head, 128 queries); it walks the keys
//                   that they see and holds dQ in TMEM.
// S and dP are computed in both, so seven products run where five would do. One
// kernel with five would add dQ up in device memory from all key blocks, 4 bytes x D
// a query and key block, with atomics (whose order changes the result) or in an
// order that CTAs wait for, and its dQ would share TMEM columns with S or dP, since
// dK, dV, dQ, S and dP of 128 x 128 x 128 tiles do not fit at once. That kernel was
// not built: this is an argument, not a measurement. With two kernels no sum is
// atomic, and results are the same from run to run.
//
// Roles of a CTA (576 threads): warps 0-15 take the S and dP tiles from TMEM and
// put P and dS back in 16 bits (four warpgroups of 32 columns each; a warp's
// lanes are 32 rows), warp 16 issues the products, warp 17 the loads. Eight such
// warps could not hide their own latencies (8 x 4096 causal tokens of 32 / 8 heads:
// 3893 us with eight, 3496 with sixteen and the elected issuer below).
//
// Five of a CTA's 18 warps share a quarter of the SM's registers, 96 a thread, and
// some values spill: at D = 128 in bf16 bwd_dq_kernel stores 84 bytes a thread and
// loads 64 (148 and 168 with a mask, 92 and 140 in parts), bwd_dkv_kernel 24 and 56
// (none with a mask, 40 and 80 in parts).
//
// Over long walks at D = 128 both are bound by the tensor cores: four (three)
// products of 512 cycles stand against one exponential a pair (512 cycles of the SM's
// 32 a cycle). Over short walks and at D = 64 they are bound by the warps' chain from
// S to dS, a block at a time, and by the tiles' ends (the tensor pipe is busy for 51%
// and 65% of the time with 8.5 blocks a tile, at D = 64 for 27% and 37% with 11 and 7:
// about 2800 and 3000 cycles a block, ends included).
// bwd_dq_kernel's products alone, in this order, take 2030 cycles a block, since
// shared memory feeds two operands of each S and dP. Measured with all they wait
// for: 2490 cycles a block where a tile has 16 of them, 3330 at 8; bwd_dkv_kernel
// 2730 at 66, 3440 at 8 (delta and the results' stores stand between two tiles).
// 8 x 4096 tokens take 2590 to 2640 us: the seven products run at 1.46 to 1.49 PFLOP/s,
// near what the tensor cores keep up at the clock that power leaves them in so long a
// call (1.73 PFLOP/s for a library product); the five that are the work at 1.05.
//
// delta and the log-sum-exp in log2 units, negated, are left for the other kernel by bwd_dq_kernel, which has dO at hand: as
// (B, Hq, Sp) with the rows of a head next to each other and padded to whole blocks, so that 128 of them are one bulk copy.
// Rows that are none, and rows without a visible key (lse = -inf), get -inf: their probabilities become 2^-inf = 0. With an
// additive mask -(row maximum) or -lse and 1 / (row sum) or 1 are left instead, and those rows get 0 and 0: the factor of 0 makes
// their probabilities 0, beside logits that must stay finite or -inf.
//
// P enters its product in the inputs' 16-bit type, as in the forward pass, and
// so does dS: the tensor cores take both operands in one type. Each is rounded
// once, from FP32, so that a term is off by half a step of that type, as the
// inputs themselves are; sums are FP32. fp16 has normal numbers from 2^-14 to 2^16
// only. Over thousands of keys most of P and dS lie below; with a scaled loss dS may
// lie above where the gradients do not. P enters as 2^14 P, and dS as 2^s dS with
// the largest s that keeps |dS| <= 2 |dO_i| max_j |v_j| (norms of head vectors) within
// 2^15 (-26 to 40), for each (b, K/V head) from its largest norms, which a pass over
// dO and V ahead finds; the powers are taken back from the sums. (dV's error over 32000 keys: 4.4e-4 without, 3.0e-4
// so, like dQ's and dK's; 3 x 777 queries over 1301 keys, 16 heads of 64: 8 us of 90.)
#pragma once

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "bwd_params.h"
#include "e4m3.cuh"

#include <type_traits>

namespace attn {
namespace bwd {

constexpr int kGroups = 4, kCols = kBlock / kGroups;       // warpgroups of the element-wise work, columns of each
constexpr int kWarps = 4 * kGroups;
constexpr int kIssueWarp = kWarps, kLoadWarp = kWarps + 1;
constexpr int kThreads = 32 * (kWarps + 2);                // 96 registers a thread
constexpr uint32_t kRowBytes = kBlock * sizeof(float);     // 128 row statistics
constexpr float kLog2E = 1.4426950408889634f;

// ------------------------------------------------------------ shared pieces

// The 128 x D tiles: boxes of 64 columns, 128-byte rows, 128-byte swizzle.
template <int D>
struct Tile {
    static constexpr int kBoxes = D / 64;
    static constexpr int kBoxBytes = 128 * 128;
    static constexpr int kBytes = kBoxes * kBoxBytes;
};

template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int h, int row, int b) {
#pragma unroll
    for (int c = 0; c < Tile<D>::kBoxes; ++c)
        ptx::tma_load_4d(dst + c * Tile<D>::kBoxBytes, map, bar, c * 64, h, row, b);
}

// Products are issued by one elected lane of a warp that knows its index to be uniform: only so do the operands stay in uniform
// registers (65 cycles an instruction of 128 x 128 x 16; 81 behind a test of the lane's number). The tensor cores take a
// product's instructions little faster than they run them, so every cycle between two products is theirs lost, and a look at
// a barrier costs the issuing warp 100 of them beside busy warps. So what a product waits for is looked at, like all
// bookkeeping, while the product before it is half issued (follow).

// Half of D(tmem) = A B^T of two tiles, summed over the head dimension.
template <int D, bool BF16>
__device__ __forceinline__ void half_over_d(int half, uint32_t d, uint32_t a, uint32_t b) {
    constexpr uint32_t kIdesc = ptx::idesc_f16(kBlock, kBlock, BF16, false, false);
    constexpr int kSteps = D / 32;
    const uint64_t ad = ptx::sdesc_kmajor_sw128(a), bd = ptx::sdesc_kmajor_sw128(b);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int kk = half * kSteps + i;
        const uint64_t off = (uint64_t)(((kk >> 2) * Tile<D>::kBoxBytes + (kk & 3) * 32) >> 4);
        ptx::mma_ss(d, ad + off, bd + off, kIdesc, kk > 0 ? 1u : 0u);
    }
}

// Half of D(tmem) (+)= A B, A 128 x 128 in TMEM as the warpgroups leave it: 16-bit pairs, each in the first half of its own
// columns.
template <int D, bool BF16>
__device__ __forceinline__ void half_over_rows(int half, uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
    constexpr uint32_t kIdesc = ptx::idesc_f16(kBlock, D, BF16, false, true);
    constexpr int kSteps = kBlock / 32;
    const uint64_t bd = ptx::sdesc_mnmajor_sw128(b, Tile<D>::kBoxBytes);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int kk = half * kSteps + i;
        ptx::mma_ts(d, a + (uint32_t)((kk >> 1) * kCols + (kk & 1) * 8), bd + (uint64_t)((kk * 16 * 128) >> 4), kIdesc,
                    (accumulate || kk > 0) ? 1u : 0u);
    }
}

// The rest of one product and the beginning of the next, which is free to go (`seen`, the same in all lanes) or waits first.
template <typename Wait, typename Tail, typename Head>
__device__ __forceinline__ bool follow(bool seen, Wait wait, Tail tail, Head head) {
    if (seen) {
        ptx::tc_fence_after_sync();
        if (ptx::elect_one()) {
            tail();
            head();
        }
        return true;
    }
    if (ptx::elect_one()) tail();
    if (!wait()) return false;
    ptx::tc_fence_after_sync();
    if (ptx::elect_one()) head();
    return true;
}

// What was issued so far arrives on `bar` when it is done.
__device__ __forceinline__ void commit(uint32_t bar) {
    if (ptx::elect_one()) ptx::tc_commit(bar);
}

// Whether two phases are complete.
__device__ __forceinline__ bool warp_test2(uint32_t bar_a, uint32_t parity_a, uint32_t bar_b, uint32_t parity_b) {
    const bool a = ptx::mbar_test_wait(bar_a, parity_a), b = ptx::mbar_test_wait(bar_b, parity_b);
    return __all_sync(0xffffffffu, a && b);
}
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, ptx::mbar_test_wait(bar, parity));
}

__device__ __forceinline__ void load32(uint32_t taddr, float* x) {
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    ptx::tmem_ld32(taddr, r);
    ptx::tmem_ld_wait();
    ptx::reg_fence32(r);
}

// Exponents that P and dS carry in fp16 (see above). range_of fetches what the pass ahead has left of a (b, K/V head), a word a
// lane (more where heads are few); ds_shift, when it is needed, finds the exponent in it.
template <bool BF16>
constexpr int kPShift = BF16 ? 0 : 14;
template <bool BF16>
__device__ __forceinline__ uint32_t range_of(const BwdParams& p, int b, int hk) {
    if constexpr (BF16) {
        return 0u;
    } else {
        const int lane = threadIdx.x & 31;
        const unsigned int* const words = p.range + ((long long)b * p.Hkv + hk) * p.n_range;
        uint32_t m = lane < p.n_range ? __ldcg(words + lane) : 0u;
        for (int i = lane + 32; i < p.n_range; i += 32) m = __vmaxu2(m, __ldcg(words + i));
        return m;
    }
}
template <bool BF16>
__device__ __forceinline__ int ds_shift(uint32_t m) {
    if constexpr (BF16) {
        return 0;
    } else {
        // the squares of the norms, rounded up; the bound's, 4 |dO|^2 |V|^2, is below 2^e
        const uint32_t g = __reduce_max_sync(0xffffffffu, m & 0xffffu), v = __reduce_max_sync(0xffffffffu, m >> 16);
        const float bound = 4.f * __uint_as_float((g + 1u) << 16) * __uint_as_float((v + 1u) << 16);
        const int e = (int)(__float_as_uint(bound) >> 23) - 126;
        return min(40, 15 - ((e + 1) >> 1));
    }
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

template <bool BF16>
__device__ __forceinline__ uint32_t pack(float a, float b) {
    return BF16 ? ptx::pack_bf16x2(a, b) : ptx::pack_f16x2(a, b);
}

// Waits for two phases; the probes of both are under way together.
__device__ __forceinline__ bool warp_wait2(uint32_t bar_a, uint32_t parity_a, uint32_t bar_b, uint32_t parity_b, const SyncCtx& sc) {
    const bool a = ptx::mbar_try_wait(bar_a, parity_a), b = ptx::mbar_try_wait(bar_b, parity_b);
    if (__all_sync(0xffffffffu, a && b)) return true;
    return warp_wait(bar_a, parity_a, sc) && warp_wait(bar_b, parity_b, sc);
}

// A warp is through with something: one arrival for its 32 lanes.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

// The same after TMEM loads or stores, which the products issued next must find done.
__device__ __forceinline__ void warp_arrive_tmem(uint32_t bar) {
    ptx::tc_fence_before_sync();
    warp_arrive(bar);
}

// N accumulated values of a row, times `factor`, to 16 bits in device memory. `freed`: a barrier to arrive on once the last
// of them are in registers.
template <int N, bool BF16>
__device__ __forceinline__ void store_row(uint32_t taddr, uint32_t freed, uint16_t* row, float factor, bool there, bool vec8) {
#pragma unroll
    for (int c = 0; c < N; c += 32) {
        float v[32];
        uint32_t w[16];
        load32(taddr + c, v);
        if (c + 32 >= N) warp_arrive_tmem(freed);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack<BF16>(v[2 * i] * factor, v[2 * i + 1] * factor);
        if (there) {
            if (vec8) {
                ptx::st_global_v8(row + c, w);
                ptx::st_global_v8(row + c + 16, w + 8);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(row + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
        }
    }
}

// The same as FP32, of a part of a tile's walk (in pieces that leave the block's P its registers).
template <int N>
__device__ __forceinline__ void store_part(uint32_t taddr, uint32_t freed, float* row, float factor, bool there) {
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        uint32_t v[16];
        ptx::tmem_ld16(taddr + c, v);
        ptx::tmem_ld_wait();
        ptx::reg_fence16(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * factor);
        if (there) {
            ptx::st_global_v8(row + c, v);
            ptx::st_global_v8(row + c + 8, v + 8);
        }
    }
    warp_arrive_tmem(freed);
}

// The mask of a warp's 32 rows (those from `row0` on) and the kCols columns from `key0` on, a row a lane. Were each lane to read
// its own row, every load would touch 32 lines; here a load touches four rows, eight lanes with four values each, and the eight
// lanes exchange what they have in three steps. Rows and columns that are none get 0.
__device__ __forceinline__ void load_mask(float (&x)[kCols], const float* mask, int row0, int rows, int key0, int keys) {
    static_assert(kCols == 32, "eight lanes of four values");
    const int lane = threadIdx.x & 31, first = row0 + (lane & 24), col = key0 + 4 * (lane & 7);
    const float* at = mask + (size_t)first * keys + col;
    const bool vec = key0 + kCols <= keys && keys % 4 == 0 && (reinterpret_cast<uintptr_t>(mask) & 15) == 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool there = first + i < rows;
        if (vec) {
            const float4 m = there ? *reinterpret_cast<const float4*>(at + (size_t)i * keys) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[4 * i] = m.x, x[4 * i + 1] = m.y, x[4 * i + 2] = m.z, x[4 * i + 3] = m.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * i + e] = there && col + e < keys ? at[(size_t)i * keys + e] : 0.f;
        }
    }
#pragma unroll
    for (int m = 1; m < 8; m *= 2) {
        const bool upper = lane & m;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (i & (4 * m)) continue;
            const float got = __shfl_xor_sync(0xffffffffu, upper ? x[i] : x[i + 4 * m], m);
            if (upper) x[i] = got;
            else x[i + 4 * m] = got;
        }
    }
}

// One warp writes zeros over `rows` rows of D values (of a tile without a visible pair), `stride` apart.
template <int D, typename Value>
__device__ __forceinline__ void zero_rows(Value* at, long long stride, int rows) {
    constexpr int kEach = 16 / sizeof(Value), kPer = D / kEach;                        // 16-byte pieces of a row
    for (int e = threadIdx.x & 31; e < rows * kPer; e += 32)
        *reinterpret_cast<uint4*>(at + (e / kPer) * stride + kEach * (e % kPer)) = make_uint4(0u, 0u, 0u, 0u);
}

// Blocks [from, from + n) of a walk of `all` blocks that part `split` takes; part 0 is empty where the walk is.
__device__ __forceinline__ int part_from(int all, int split, int splits) {
    return min(all, split * ((all + splits - 1) / splits));
}

// Work tiles are handed out in order: a CTA's first is its own index, each further one comes from a counter in the
// workspace when the CTA is about to load it, so that CTAs with short tiles take more of them. (Which CTA computes a tile
// changes nothing in it.) The loading warp publishes them in a ring of two entries; every other warp takes a copy. Tiles
// without a visible pair are not published: the loading warp writes their zeros.
struct TileRing {
    uint32_t full, empty;           // barriers, two each
    volatile int* entry;
};
constexpr int kRing = 2;
constexpr uint32_t kRingReaders = kWarps + 1;

// Loading warp: the CTA's next tile, or -1 behind the last. `taken`: tiles taken so far.
__device__ __forceinline__ int take_tile(uint32_t& taken, const BwdParams& p) {
    int t = 0;
    if ((threadIdx.x & 31) == 0) {
        t = taken == 0 ? (int)blockIdx.x : (int)min((long long)gridDim.x + atomicAdd(p.counter, 1u), (long long)p.n_tiles);
        if (t >= p.n_tiles) t = -1;
    }
    ++taken;
    return __shfl_sync(0xffffffffu, t, 0);
}

// Loading warp: publishes tile t (-1: the end) as the ring's k-th entry. False where a wait ran out.
__device__ __forceinline__ bool publish_tile(uint32_t k, int t, const TileRing& ring, const SyncCtx& sc) {
    const uint32_t s = k % kRing;
    if (k >= kRing && !warp_wait(ring.empty + 8 * s, (k / kRing - 1) & 1u, sc)) return false;
    if ((threadIdx.x & 31) == 0) {
        ring.entry[s] = t;
        ptx::mbar_arrive(ring.full + 8 * s);
    }
    return true;
}

// The k-th entry of the ring: a tile, or -1 at the end (or where a wait ran out).
__device__ __forceinline__ int next_tile(uint32_t k, const TileRing& ring, const SyncCtx& sc) {
    const uint32_t s = k % kRing;
    if (!warp_wait(ring.full + 8 * s, (k / kRing) & 1u, sc)) return -1;
    const int t = ring.entry[s];
    warp_arrive(ring.empty + 8 * s);
    return __shfl_sync(0xffffffffu, t, 0);                    // (known to be uniform, and with it what follows from it)
}

// A place in a ring of N buffers: which buffer, and how often it was used before (its barriers' parity).
template <int N>
struct Place {
    uint32_t at = 0, round = 0;
    __device__ __forceinline__ uint32_t parity() const { return round & 1u; }
    __device__ __forceinline__ Place next() const {
        Place n = *this;
        if (++n.at == N) n.at = 0, ++n.round;
        return n;
    }
};

// ------------------------------------------------------------------ dK, dV
//
// TMEM: S^T and then P^T in columns 0-127, dP^T and then dS^T in 128-255, dV from
// 256, dK behind it. A query block i of the walk takes, in the tensor cores' order,
//   dV += P_i^T dO_i,  S_{i+1}^T = K Q_{i+1}^T,  dK += dS_i^T Q_i,  dP_{i+1}^T = V dO_{i+1}^T
// so that the warps find P's work under the last two products of a block and dS's
// under the first two. S^T of the next block overwrites P^T, whose product was
// issued before it by the same thread: the tensor cores run one thread's products
// in order. Rows are keys here, so that P^T and dS^T are operands as they stand.

template <int D, bool ADDITIVE>
struct KvCfg {
    using T = Tile<D>;
    // Q stays until the last product of its block, dO until the first.
    static constexpr int kQ = D == 128 ? (ADDITIVE ? 2 : 3) : 5, kG = D == 128 ? 2 : 4;
    static constexpr int kKOff = 0, kVOff = T::kBytes, kQOff = 2 * T::kBytes, kGOff = kQOff + kQ * T::kBytes;
    static constexpr int kRowOff = kGOff + kG * T::kBytes;                  // [kQ] -lse, [kG] -delta, [kQ] 1 / sum
    static constexpr int kDeltaOff = kRowOff + kQ * (int)kRowBytes;
    static constexpr int kSumOff = kDeltaOff + kG * (int)kRowBytes;
    static constexpr int kBarOff = kSumOff + (ADDITIVE ? kQ * (int)kRowBytes : 0);
    static constexpr int bK = 0, bV = 1, bKEmpty = 2, bVEmpty = 3, bP = 4, bDS = 5, bAcc = 6, bAccEmpty = 7, bDrain = 8,
                         bStall = 9, bS = 10, bDP = 11, bTile = 12, bTileEmpty = bTile + kRing, bQ = bTileEmpty + kRing, bQEmpty = bQ + kQ,
                         bG = bQEmpty + kQ, bGEmpty = bG + kG, kNumBars = bGEmpty + kG;
    static constexpr int kTmemSlotOff = kBarOff + 8 * kNumBars;
    static constexpr int kAbortOff = kTmemSlotOff + 4;
    static constexpr int kTileOff = kAbortOff + 4;
    static constexpr int kSmemBytes = kTileOff + 4 * kRing;
    static constexpr uint32_t cS = 0, cDP = 128, cDV = 256, cDK = 256 + D;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct KvTile {
    int b, hk, k0;
    int lo, per_head;       // first query block that sees a key of the tile, and how many do
    int split, from, n;     // part of the walk over the blocks of every head (-1: whole), its first block and how many
};

// Tiles of a K/V head follow each other, so that its queries come from L2; with a causal mask the first keys, which most
// queries see, come first. A window's sinks are seen by all queries: their tiles, the longest, come before all others (16384
// tokens, 8 K/V heads, window 4096, 4 sinks: 2634 us with them at the head of each K/V head's tiles, 2104 so).
template <bool PARTS>
__device__ __forceinline__ KvTile kv_tile(int t, const BwdParams& p) {
    KvTile w;
    w.split = -1;
    if (PARTS) {
        const int parts = p.cut * p.splits;
        w.split = t < parts ? t % p.splits : -1;
        t = t < parts ? t / p.splits : t - parts + p.cut;
    }
    const int sinks = p.sink_kb * p.B * p.Hkv;                 // tiles
    const bool sink = t < sinks;
    const int of = sink ? p.sink_kb : p.n_kb - p.sink_kb, at = sink ? t : t - sinks, bh = at / max(of, 1);
    w.k0 = (at - bh * of + (sink ? 0 : p.sink_kb)) * kBlock;
    w.b = bh / p.Hkv;
    w.hk = bh - w.b * p.Hkv;
    int lo = 0, hi = p.Sq;                                     // queries
    if (p.causal) lo = max(0, w.k0 - p.off);
    if (p.window && w.k0 >= p.sinks) hi = (int)min((long long)p.Sq, (long long)w.k0 + kBlock - 1 - p.off + p.window);
    w.lo = lo / kBlock;
    w.per_head = hi > lo ? (hi + kBlock - 1) / kBlock - w.lo : 0;
    w.n = w.per_head * p.group;
    w.from = 0;
    if (PARTS && w.split >= 0) {
        w.from = part_from(w.n, w.split, p.splits);
        w.n = part_from(w.n, w.split + 1, p.splits) - w.from;
    }
    return w;
}

template <int D, bool BF16, bool ADDITIVE, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG, const BwdParams p) {
    using C = KvCfg<D, ADDITIVE>;
    using T = Tile<D>;
    extern __shared__ __align__(1024) uint8_t smem_ptr[];
    const uint32_t smem = ptx::smem_addr(smem_ptr);
    if (smem & 1023u) {                               // swizzled tiles: the linker aligns the array, never seen otherwise
        if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (known to be uniform)
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem_ptr + C::kAbortOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_ptr + C::kTmemSlotOff);
    auto bar = [&](int i) { return smem + C::kBarOff + 8u * (uint32_t)i; };
    const TileRing ring{bar(C::bTile), bar(C::bTileEmpty), reinterpret_cast<volatile int*>(smem_ptr + C::kTileOff)};

    if (warp == kLoadWarp && lane == 0) {
        for (int i = 0; i < C::kNumBars; ++i) {
            uint32_t count = 1;
            if (i >= C::bTileEmpty && i < C::bTileEmpty + kRing) count = kRingReaders;
            if (i == C::bP || i == C::bDS || i == C::bAccEmpty) count = kWarps;
            // a block's tile is free once its last product has run and the warps have its statistics
            if ((i >= C::bQEmpty && i < C::bQEmpty + C::kQ) || (i >= C::bGEmpty && i < C::bGEmpty + C::kG)) count = kWarps + 1;
            ptx::mbar_init(bar(i), count);
        }
        *abort_flag = 0u;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_shared();
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
        ptx::prefetch_tensormap(&tmG);
    }
    if (warp == kIssueWarp) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const SyncCtx sc{abort_flag, p.status, p.timeout_ns};
    wait_for_inputs();                                // nothing above touches global memory
    let_next_start();

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        uint32_t taken = 0, tiles = 0, v_fills = 0, q_fills = 0, g_fills = 0;
        Place<C::kQ> q;
        Place<C::kG> g;
        for (bool alive = true; alive;) {
            const int t = take_tile(taken, p);
            const KvTile w = kv_tile<PARTS>(max(t, 0), p);
            if (t >= 0 && w.n == 0) {
                const long long token = (long long)w.b * p.Sk + w.k0;
                const int rows = min(kBlock, p.Sk - w.k0);
                if (PARTS && w.split >= 0) {
                    const long long plane = (long long)p.B * p.part_rows * p.Hkv * D;
                    float* part = p.part + 2 * w.split * plane + (((long long)w.b * p.part_rows + w.k0) * p.Hkv + w.hk) * D;
                    zero_rows<D>(part, (long long)p.Hkv * D, rows);
                    zero_rows<D>(part + plane, (long long)p.Hkv * D, rows);
                    continue;
                }
                zero_rows<D>(static_cast<uint16_t*>(p.dk) + token * p.dk_stride + w.hk * D, p.dk_stride, rows);
                zero_rows<D>(static_cast<uint16_t*>(p.dv) + token * p.dv_stride + w.hk * D, p.dv_stride, rows);
                continue;
            }
            if (!publish_tile(tiles, t, ring, sc) || t < 0) break;
            if (tiles > 0 && !warp_wait(bar(C::bKEmpty), (tiles - 1) & 1u, sc)) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(bar(C::bK), T::kBytes);
                load_tile<D>(smem + C::kKOff, &tmK, bar(C::bK), w.hk, w.k0, w.b);
            }
            ++tiles;
            int h = w.hk * p.group + (PARTS ? w.from / w.per_head : 0), i = w.lo + (PARTS ? w.from % w.per_head : 0);
            for (int it = 0; it < w.n; ++it) {
                const size_t row = ((size_t)w.b * p.Hq + h) * p.Sp + (size_t)i * kBlock;
                if (q.round > 0 && !(alive = warp_wait(bar(C::bQEmpty + q.at), (q.round - 1) & 1u, sc))) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(C::bQ + q.at), T::kBytes + kRowBytes * (ADDITIVE ? 2 : 1));
                    load_tile<D>(smem + C::kQOff + q.at * T::kBytes, &tmQ, bar(C::bQ + q.at), h, i * kBlock, w.b);
                    ptx::bulk_load(smem + C::kRowOff + q.at * kRowBytes, p.neg_lse + row, kRowBytes, bar(C::bQ + q.at));
                    if (ADDITIVE)
                        ptx::bulk_load(smem + C::kSumOff + q.at * kRowBytes, p.inv_sum + row, kRowBytes, bar(C::bQ + q.at));
                }
                ++q_fills;
                q = q.next();
                if (g.round > 0 && !(alive = warp_wait(bar(C::bGEmpty + g.at), (g.round - 1) & 1u, sc))) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(C::bG + g.at), T::kBytes + kRowBytes);
                    load_tile<D>(smem + C::kGOff + g.at * T::kBytes, &tmG, bar(C::bG + g.at), h, i * kBlock, w.b);
                    ptx::bulk_load(smem + C::kDeltaOff + g.at * kRowBytes, p.neg_delta + row, kRowBytes, bar(C::bG + g.at));
                }
                ++g_fills;
                g = g.next();
                if (it == 0) {
                    if (v_fills > 0 && !(alive = warp_wait(bar(C::bVEmpty), (v_fills - 1) & 1u, sc))) break;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bar(C::bV), T::kBytes);
                        load_tile<D>(smem + C::kVOff, &tmV, bar(C::bV), w.hk, w.k0, w.b);
                    }
                    ++v_fills;
                }
                if (++i == w.lo + w.per_head) {
                    i = w.lo;
                    ++h;
                }
            }
        }
        // Shut down: every copy has landed.
        if (tiles > 0) drain_phase(bar(C::bK), (tiles - 1) & 1u, sc);
        if (v_fills > 0) drain_phase(bar(C::bV), (v_fills - 1) & 1u, sc);
        for (uint32_t s = 0; s < (uint32_t)C::kQ; ++s)
            if (q_fills > s) drain_phase(bar(C::bQ + s), ((q_fills - 1 - s) / C::kQ) & 1u, sc);
        for (uint32_t s = 0; s < (uint32_t)C::kG; ++s)
            if (g_fills > s) drain_phase(bar(C::bG + s), ((g_fills - 1 - s) / C::kG) & 1u, sc);
    } else if (warp == kIssueWarp) {
        // --------------------------------------------------------- products
        // One walk over the blocks of all tiles: a tile's first S and dP are issued before the last tile's last dK.
        uint32_t k = 0, tiles = 0, use = 0;                   // ring entries, tiles done, blocks
        Place<C::kQ> q;
        Place<C::kG> g;
        bool alive = true, issued = false;
        // Blocks of the next tile; 0: there is none.
        auto next_work = [&]() -> int {
            const int t = next_tile(k++, ring, sc);
            return t < 0 ? 0 : kv_tile<PARTS>(t, p).n;
        };
        auto s_half = [&](int half, uint32_t at) {
            half_over_d<D, BF16>(half, tmem + C::cS, smem + C::kKOff, smem + C::kQOff + at * T::kBytes);
        };
        auto dp_half = [&](int half, uint32_t at) {
            half_over_d<D, BF16>(half, tmem + C::cDP, smem + C::kVOff, smem + C::kGOff + at * T::kBytes);
        };
        if (p.stall) alive = warp_wait(bar(C::bStall), 0, sc);               // nothing ever arrives
        int n = alive ? next_work() : 0, it = 0;
        if (n > 0) {
            alive = warp_wait2(bar(C::bK), 0, bar(C::bQ + q.at), q.parity(), sc);
            if (alive) {
                issued = true;
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) {
                    s_half(0, q.at);
                    s_half(1, q.at);
                    ptx::tc_commit(bar(C::bS));
                    if (n == 1) ptx::tc_commit(bar(C::bKEmpty));
                }
                alive = warp_wait2(bar(C::bV), 0, bar(C::bG + g.at), g.parity(), sc);
            }
            if (alive) {
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) dp_half(0, g.at);
            }
        }
        while (alive && n > 0) {
            // (dP of this block is half issued)
            const bool last = it + 1 == n, drained = it > 0 || tiles == 0;
            const uint32_t acc_parity = (tiles - 1) & 1u;     // the warps have the last tile's dK and dV
            alive = follow(
                drained ? warp_test(bar(C::bP), use & 1u)
                        : warp_test2(bar(C::bP), use & 1u, bar(C::bAccEmpty), acc_parity),
                [&] { return warp_wait(bar(C::bP), use & 1u, sc) && (drained || warp_wait(bar(C::bAccEmpty), acc_parity, sc)); },
                [&] {
                    dp_half(1, g.at);
                    ptx::tc_commit(bar(C::bDP));
                    if (last) ptx::tc_commit(bar(C::bVEmpty));
                },
                [&] { half_over_rows<D, BF16>(0, tmem + C::cDV, tmem + C::cS, smem + C::kGOff + g.at * T::kBytes, it > 0); });
            if (!alive) break;
            auto dv_rest = [&] {
                half_over_rows<D, BF16>(1, tmem + C::cDV, tmem + C::cS, smem + C::kGOff + g.at * T::kBytes, true);
                ptx::tc_commit(bar(C::bGEmpty + g.at));
            };
            auto dk_begin = [&] {
                half_over_rows<D, BF16>(0, tmem + C::cDK, tmem + C::cDP, smem + C::kQOff + q.at * T::kBytes, it > 0);
            };
            auto dk_rest = [&] {
                half_over_rows<D, BF16>(1, tmem + C::cDK, tmem + C::cDP, smem + C::kQOff + q.at * T::kBytes, true);
                ptx::tc_commit(bar(C::bQEmpty + q.at));
                if (last) ptx::tc_commit(bar(C::bAcc));
            };
            auto wait_ds = [&] { return warp_wait(bar(C::bDS), use & 1u, sc); };
            // the block after this one: number i1 of n1 of its tile
            const Place<C::kQ> q1 = q.next();
            const Place<C::kG> g1 = g.next();
            const int n1 = last ? next_work() : n, i1 = last ? 0 : it + 1;
            if (n1 == 0) {
                alive = follow(false, wait_ds, dv_rest, [&] { dk_begin(); dk_rest(); });
                break;
            }
            const uint32_t kv_parity = (tiles + 1) & 1u;      // of a new tile's K and V
            alive = follow(
                last ? warp_test2(bar(C::bQ + q1.at), q1.parity(), bar(C::bK), kv_parity) : warp_test(bar(C::bQ + q1.at), q1.parity()),
                [&] { return warp_wait(bar(C::bQ + q1.at), q1.parity(), sc) && (!last || warp_wait(bar(C::bK), kv_parity, sc)); },
                dv_rest, [&] { s_half(0, q1.at); });
            if (!alive) break;
            alive = follow(
                warp_test(bar(C::bDS), use & 1u), wait_ds,
                [&] {
                    s_half(1, q1.at);
                    ptx::tc_commit(bar(C::bS));
                    if (i1 + 1 == n1) ptx::tc_commit(bar(C::bKEmpty));
                },
                dk_begin);
            if (!alive) break;
            alive = follow(
                last ? warp_test2(bar(C::bG + g1.at), g1.parity(), bar(C::bV), kv_parity) : warp_test(bar(C::bG + g1.at), g1.parity()),
                [&] { return warp_wait(bar(C::bG + g1.at), g1.parity(), sc) && (!last || warp_wait(bar(C::bV), kv_parity, sc)); },
                dk_rest, [&] { dp_half(0, g1.at); });
            tiles += last;
            n = n1;
            it = i1;
            ++use;
            q = q1;
            g = g1;
        }
        if (issued) {                                         // TMEM is freed after every product has run
            if (ptx::elect_one()) ptx::tc_commit(bar(C::bDrain));
            drain_phase(bar(C::bDrain), 0, sc);
        }
        __syncwarp();
    } else if (warp < kWarps) {
        // ------------------------------------------------------- P^T and dS^T
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane;     // key of the tile; columns kCols wg ..
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + C::cS + kCols * wg, tDP = tmem + lane_base + C::cDP + kCols * wg;
        const float sl = p.scale_log2;
        int shift = 0;                                               // of the tile
        float more = 1.f, back = 1.f;                                // of dS over P; of the tile before
        uint32_t tiles = 0, use = 0;
        Place<C::kQ> q;
        Place<C::kG> g;
        bool alive = true;
        // Two warpgroups write dV, two dK, each half of the row: of the tile before, once the first P of the next one is done
        const bool is_k = wg >= 2;
        const int col = (wg & 1) * (D / 2);
        void* done_row = nullptr;
        bool done_there = false, done_part = false;
        auto finish = [&]() -> bool {
            if (!done_row) return true;
            if (!warp_wait(bar(C::bAcc), tiles & 1u, sc)) return false;
            ptx::tc_fence_after_sync();
            const uint32_t acc = tmem + lane_base + (is_k ? C::cDK : C::cDV) + col;
            if (PARTS && done_part)
                store_part<D / 2>(acc, bar(C::bAccEmpty), static_cast<float*>(done_row), back, done_there);
            else
                store_row<D / 2, BF16>(acc, bar(C::bAccEmpty), static_cast<uint16_t*>(done_row), is_k ? p.scale * back : back, done_there,
                                       p.vec8);
            done_row = nullptr;
            ++tiles;
            return true;
        };
        for (uint32_t k = 0; alive; ++k) {
            const int t = next_tile(k, ring, sc);
            if (t < 0) break;
            const KvTile w = kv_tile<PARTS>(t, p);
            const uint32_t range = range_of<BF16>(p, w.b, w.hk);
            const int key = w.k0 + r;
            // queries [see, end) see this key
            const int see = p.causal ? key - p.off : 0;
            const int end = p.window && key >= p.sinks
                                ? (int)min((long long)INT_MAX, (long long)key - p.off + p.window) : INT_MAX;
            // blocks that begin at or after all_see and end at or before all_end hide nothing
            const int all_see = p.causal ? w.k0 + kBlock - 1 - p.off : 0;
            const int all_end = p.window && w.k0 + kBlock > p.sinks
                                    ? (int)min((long long)INT_MAX, (long long)max(w.k0, p.sinks) - p.off + p.window) : INT_MAX;
            int i = w.lo + (PARTS ? w.from % w.per_head : 0);
            for (int it = 0; it < w.n; ++it, ++use, q = q.next(), g = g.next()) {
                const int m0 = i * kBlock + kCols * wg;              // this warp's first query
                float x[kCols];
                if (ADDITIVE) {
                    // a warp's lanes are neighbouring keys: each load is one line of the mask
                    const float* at = p.mask + ((size_t)w.b * p.Sq + m0) * p.Sk + key;
#pragma unroll
                    for (int c = 0; c < kCols; ++c) x[c] = (key < p.Sk && m0 + c < p.Sq) ? at[(size_t)c * p.Sk] : 0.f;
                }
                if (!(alive = warp_wait(bar(C::bQ + q.at), q.parity(), sc))) break;
                const float4* nl = reinterpret_cast<const float4*>(smem_ptr + C::kRowOff + q.at * kRowBytes) + kCols / 4 * wg;
                if (ADDITIVE) {
                    if (!(alive = warp_wait(bar(C::bS), use & 1u, sc))) break;
                    ptx::tc_fence_after_sync();
                    const float4* is = reinterpret_cast<const float4*>(smem_ptr + C::kSumOff + q.at * kRowBytes) + kCols / 4 * wg;
                    float s[kCols];
                    load32(tS, s);
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) {
                        const float4 n = nl[c / 4], u = is[c / 4];
                        const float nn[4] = {n.x, n.y, n.z, n.w}, uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            float y = fmaf(x[c + d], kLog2E, s[c + d] * sl);
                            if (m0 + c + d < see) y = -INFINITY;
                            x[c + d] = ptx::ex2(y + nn[d]) * uu[d];
                        }
                    }
                } else {
                    float s[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) {
                        const float4 n = nl[c / 4];
                        x[c] = n.x, x[c + 1] = n.y, x[c + 2] = n.z, x[c + 3] = n.w;
                    }
                    if (!(alive = warp_wait(bar(C::bS), use & 1u, sc))) break;
                    ptx::tc_fence_after_sync();
                    load32(tS, s);
#pragma unroll
                    for (int c = 0; c < kCols; c += 2) ptx::fma2(x[c], x[c + 1], s[c], s[c + 1], sl, sl, x[c], x[c + 1]);
                    const int base = i * kBlock;
                    if (base < all_see || base > all_end - kBlock) {
                        const int c0 = see - m0, c1 = end - m0;
#pragma unroll
                        for (int c = 0; c < kCols; ++c)
                            if (c < c0 || c >= c1) x[c] = -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < kCols; ++c) x[c] = ptx::ex2(x[c]);
                }
                {
                    uint32_t pk[kCols / 2];
#pragma unroll
                    for (int c = 0; c < kCols / 2; ++c) pk[c] = pack<BF16>(x[2 * c], x[2 * c + 1]);
                    ptx::tmem_st16(tS, pk);
                    ptx::tmem_st_wait();
                }
                warp_arrive_tmem(bar(C::bP));
                if (lane == 0) ptx::mbar_arrive(bar(C::bQEmpty + q.at));
                if (it == 0) {
                    if (!(alive = finish())) break;
                    shift = ds_shift<BF16>(range);
                    more = power_of_two(shift - kPShift<BF16>);
                }
                // ---- dS = P (dP - delta)
                alive = warp_wait2(bar(C::bG + g.at), g.parity(), bar(C::bDP), use & 1u, sc);
                if (!alive) break;
                ptx::tc_fence_after_sync();
                const float4* nd = reinterpret_cast<const float4*>(smem_ptr + C::kDeltaOff + g.at * kRowBytes) + kCols / 4 * wg;
                {
                    float d[kCols];
                    uint32_t pk[kCols / 2];
                    load32(tDP, d);
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) {
                        const float4 n = nd[c / 4];
                        if (BF16) {
                            ptx::add2(d[c], d[c + 1], d[c], d[c + 1], n.x, n.y);
                            ptx::add2(d[c + 2], d[c + 3], d[c + 2], d[c + 3], n.z, n.w);
                        } else {                              // (delta comes with that factor)
                            ptx::fma2(d[c], d[c + 1], d[c], d[c + 1], more, more, n.x, n.y);
                            ptx::fma2(d[c + 2], d[c + 3], d[c + 2], d[c + 3], more, more, n.z, n.w);
                        }
                        ptx::mul2(d[c], d[c + 1], d[c], d[c + 1], x[c], x[c + 1]);
                        ptx::mul2(d[c + 2], d[c + 3], d[c + 2], d[c + 3], x[c + 2], x[c + 3]);
                        pk[c / 2] = pack<BF16>(d[c], d[c + 1]);
                        pk[c / 2 + 1] = pack<BF16>(d[c + 2], d[c + 3]);
                    }
                    ptx::tmem_st16(tDP, pk);
                    ptx::tmem_st_wait();
                }
                warp_arrive_tmem(bar(C::bDS));
                if (lane == 0) ptx::mbar_arrive(bar(C::bGEmpty + g.at));
                if (++i == w.lo + w.per_head) i = w.lo;
            }
            if (!alive) break;
            const long long token = (long long)w.b * p.Sk + key;
            void* row = static_cast<uint16_t*>(is_k ? p.dk : p.dv) + token * (is_k ? p.dk_stride : p.dv_stride) + w.hk * D + col;
            if (PARTS && w.split >= 0)
                row = p.part + (2 * w.split + is_k) * ((long long)p.B * p.part_rows * p.Hkv * D) +
                      (((long long)w.b * p.part_rows + key) * p.Hkv + w.hk) * D + col;
            done_part = PARTS && w.split >= 0;
            done_row = row;
            done_there = key < p.Sk;
            back = power_of_two(is_k ? -shift : -kPShift<BF16>);
        }
        if (alive) finish();
    }

    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kIssueWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------- dQ
//
// TMEM: dQ from column 0, S of even blocks of the walk and then their dS in
// 128-255, of odd blocks in 256-383, dP in 384-511. A key block j takes, in the
// tensor cores' order,
//   dP_{j+1} = dO V_{j+1}^T,  dQ += dS_j K_j,  S_{j+2} = Q K_{j+2}^T
// the first once the warps hold dP_j in registers, the second once they have left
// dS_j. (One dP and two S: the warps' next exponentials need not wait for anything.
// S and dP in one another's columns, or Q held in TMEM, cost 6 to 13%.)
//
// With an additive mask the block's 64 KB of mask, which every head reads again from
// L2, bound both kernels: they stand in front of its exponentials, and what K, V,
// Q and dO leave of shared memory and registers does not hold them a block ahead
// (2 x 2048 tokens of 16 heads of 128: 5900 cycles a block, 329 us).

// With an additive mask a tile's keys are walked once where its rows' lse are in this range, whose rounding moves a
// probability by 2^-16 of itself, little beside that to 16 bits; else twice: a mask of large values leaves lse without the
// logits' bits, and the rows' maximum and sum are found anew.
constexpr float kPlainLse = 256.f;

// Ring entry of a tile that is walked twice.
__device__ __forceinline__ int twice_entry(int t) { return -2 - t; }

template <int D, bool ADDITIVE>
struct QCfg {
    using T = Tile<D>;
    // K stays from its S to its dQ, two blocks later
    static constexpr int kK = D == 128 ? 3 : 5, kV = D == 128 ? (ADDITIVE ? 1 : 2) : 4;
    static constexpr int kQOff = 0, kGOff = T::kBytes, kKOff = 2 * T::kBytes, kVOff = kKOff + kK * T::kBytes;
    static constexpr int kBarOff = kVOff + kV * T::kBytes;
    static constexpr int bQ = 0, bQEmpty = 1, bS = 2, bDP = 4, bDPFree = 5, bDS = 6, bAcc = 8, bAccEmpty = 9, bDrain = 10,
                         bStall = 11, bParts = 12, bWhole = 13, bG = 14, bGEmpty = 15, bDelta = 16, bTile = 17,
                         bTileEmpty = bTile + kRing, bK = bTileEmpty + kRing, bKEmpty = bK + kK, bV = bKEmpty + kK, bVEmpty = bV + kV,
                         kNumBars = bVEmpty + kV;
    static constexpr int kTmemSlotOff = kBarOff + 8 * kNumBars;
    static constexpr int kAbortOff = kTmemSlotOff + 4;
    static constexpr int kTileOff = kAbortOff + 4;
    static constexpr int kStatOff = (kTileOff + 4 * kRing + 15) / 16 * 16;      // additive mask: [kGroups][128] {maximum, sum}
    static constexpr int kDeltaOff = kStatOff + (ADDITIVE ? kGroups * 128 * 8 : 0);       // [128] -delta
    static constexpr int kSmemBytes = kDeltaOff + 128 * 4;
    static constexpr uint32_t cDQ = 0, cS = 128, cDP = 384;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct QTile {
    int b, h, hk, m0;
    int first, gap;         // key blocks of the walk: 0 .. first - 1 (sinks), then on from first + gap
    int split, from, n;     // part of the walk, its first block and how many
    __device__ __forceinline__ int block(int j) const { return j + from < first ? j + from : j + from + gap; }    // (from 0: whole)
};

// Tiles of a head follow each other; with a causal mask the last queries, which see most keys, come first.
template <bool PARTS>
__device__ __forceinline__ QTile q_tile(int t, const BwdParams& p) {
    QTile w;
    w.split = 0;
    if (PARTS) {
        w.split = t % p.splits;
        t /= p.splits;
    }
    const int bh = t / p.n_qb, m = t - bh * p.n_qb;
    w.m0 = (p.causal ? p.n_qb - 1 - m : m) * kBlock;
    w.b = bh / p.Hq;
    w.h = bh - w.b * p.Hq;
    w.hk = w.h / p.group;
    int hi = p.Sk;
    if (p.causal) hi = min(p.Sk, max(0, min(w.m0 + kBlock, p.Sq) + p.off));
    w.n = (hi + kBlock - 1) / kBlock;
    w.first = w.gap = 0;
    if (p.window) {
        const int low = max(0, w.m0 + p.off - p.window + 1) / kBlock, sinks = (min(p.sinks, hi) + kBlock - 1) / kBlock;
        if (low > sinks && low <= w.n) {
            w.first = sinks;
            w.gap = low - sinks;
            w.n -= w.gap;
        }
    }
    w.from = 0;
    if (PARTS) {
        w.from = part_from(w.n, w.split, p.splits);
        w.n = part_from(w.n, w.split + 1, p.splits) - w.from;
    }
    return w;
}

template <int D, bool BF16, bool ADDITIVE, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG, const BwdParams p) {
    using C = QCfg<D, ADDITIVE>;
    using T = Tile<D>;
    extern __shared__ __align__(1024) uint8_t smem_ptr[];
    const uint32_t smem = ptx::smem_addr(smem_ptr);
    if (smem & 1023u) {                               // swizzled tiles: the linker aligns the array, never seen otherwise
        if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (known to be uniform)
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem_ptr + C::kAbortOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_ptr + C::kTmemSlotOff);
    auto bar = [&](int i) { return smem + C::kBarOff + 8u * (uint32_t)i; };
    const TileRing ring{bar(C::bTile), bar(C::bTileEmpty), reinterpret_cast<volatile int*>(smem_ptr + C::kTileOff)};

    if (warp == kLoadWarp && lane == 0) {
        for (int i = 0; i < C::kNumBars; ++i) {
            uint32_t count = 1;
            if (i >= C::bTileEmpty && i < C::bTileEmpty + kRing) count = kRingReaders;
            if (i == C::bDPFree || i == C::bDS || i == C::bDS + 1 || i == C::bAccEmpty || i == C::bDelta) count = kWarps;
            if (i == C::bGEmpty) count = kWarps + 1;              // the last dP has run, and the warps have delta
            if (i == C::bParts) count = kWarps - 4;
            if (i == C::bWhole) count = 4;
            ptx::mbar_init(bar(i), count);
        }
        *abort_flag = 0u;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_shared();
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
        ptx::prefetch_tensormap(&tmG);
    }
    if (warp == kIssueWarp) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const SyncCtx sc{abort_flag, p.status, p.timeout_ns};
    wait_for_inputs();                                // nothing above touches global memory
    let_next_start();

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        uint32_t taken = 0, tiles = 0, g_fills = 0, kf = 0, vf = 0;
        for (bool alive = true; alive;) {
            const int t = take_tile(taken, p);
            const QTile w = q_tile<PARTS>(max(t, 0), p);
            if (t >= 0 && w.n == 0) {
                const long long token = (long long)w.b * p.Sq + w.m0;
                if (PARTS)
                    zero_rows<D>(p.part + w.split * ((long long)p.B * p.Sq * p.Hq * D) + (token * p.Hq + w.h) * D,
                                 (long long)p.Hq * D, min(kBlock, p.Sq - w.m0));
                else
                    zero_rows<D>(static_cast<uint16_t*>(p.dq) + token * p.dq_stride + w.h * D, p.dq_stride,
                                 min(kBlock, p.Sq - w.m0));
                if (w.split > 0) continue;
                // the other kernel passes over these rows too
                const size_t at = ((size_t)w.b * p.Hq + w.h) * p.Sp + w.m0;
                for (int e = lane; e < kBlock; e += 32) {
                    p.neg_delta[at + e] = 0.f;
                    p.neg_lse[at + e] = ADDITIVE ? 0.f : -INFINITY;
                    if (ADDITIVE) p.inv_sum[at + e] = 0.f;
                }
                continue;
            }
            bool twice = false;
            if (ADDITIVE && t >= 0) {
                for (int e = lane; e < min(kBlock, p.Sq - w.m0); e += 32) {
                    const float l = p.lse[((size_t)w.b * p.Hq + w.h) * p.Sq + w.m0 + e];
                    twice |= !(fabsf(l) <= kPlainLse) && l != -INFINITY;
                }
                twice = __any_sync(0xffffffffu, twice);
            }
            if (!publish_tile(tiles, twice ? twice_entry(t) : t, ring, sc) || t < 0) break;
            for (int e = lane; e < min(kBlock, p.Sq - w.m0); e += 32) {       // O, for delta: on its way to L2
                const char* o = reinterpret_cast<const char*>(p.o + (((size_t)w.b * p.Sq + w.m0 + e) * p.Hq + w.h) * D);
#pragma unroll
                for (int c = 0; c < 2 * D; c += 128) ptx::prefetch_l2(o + c);
            }
            if (tiles > 0 && !warp_wait(bar(C::bQEmpty), (tiles - 1) & 1u, sc)) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(bar(C::bQ), T::kBytes);
                load_tile<D>(smem + C::kQOff, &tmQ, bar(C::bQ), w.h, w.m0, w.b);
            }
            ++tiles;
            auto load_g = [&]() -> bool {
                if (g_fills > 0 && !warp_wait(bar(C::bGEmpty), (g_fills - 1) & 1u, sc)) return false;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(C::bG), T::kBytes);
                    load_tile<D>(smem + C::kGOff, &tmG, bar(C::bG), w.h, w.m0, w.b);
                }
                ++g_fills;
                return true;
            };
            auto load_k = [&](int j) -> bool {
                const uint32_t s = kf % C::kK;
                if (kf >= (uint32_t)C::kK && !warp_wait(bar(C::bKEmpty + s), (kf / C::kK - 1) & 1u, sc)) return false;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(C::bK + s), T::kBytes);
                    load_tile<D>(smem + C::kKOff + s * T::kBytes, &tmK, bar(C::bK + s), w.hk, w.block(j) * kBlock, w.b);
                }
                ++kf;
                return true;
            };
            auto load_v = [&](int j) -> bool {
                const uint32_t s = vf % C::kV;
                if (vf >= (uint32_t)C::kV && !warp_wait(bar(C::bVEmpty + s), (vf / C::kV - 1) & 1u, sc)) return false;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(C::bV + s), T::kBytes);
                    load_tile<D>(smem + C::kVOff + s * T::kBytes, &tmV, bar(C::bV + s), w.hk, w.block(j) * kBlock, w.b);
                }
                ++vf;
                return true;
            };
            if (twice)
                for (int j = 0; j < w.n && alive; ++j) alive = load_k(j);
            // in the order in which the products take them: K_0, dO, V_0, K_1, V_1, ...
            for (int j = 0; j < w.n && alive; ++j) alive = load_k(j) && (j > 0 || load_g()) && load_v(j);
        }
        if (tiles > 0) drain_phase(bar(C::bQ), (tiles - 1) & 1u, sc);
        if (g_fills > 0) drain_phase(bar(C::bG), (g_fills - 1) & 1u, sc);
        for (uint32_t s = 0; s < (uint32_t)C::kK; ++s)
            if (kf > s) drain_phase(bar(C::bK + s), ((kf - 1 - s) / C::kK) & 1u, sc);
        for (uint32_t s = 0; s < (uint32_t)C::kV; ++s)
            if (vf > s) drain_phase(bar(C::bV + s), ((vf - 1 - s) / C::kV) & 1u, sc);
    } else if (warp == kIssueWarp) {
        // --------------------------------------------------------- products
        // One walk over the blocks of all tiles (those walked twice have `skip` blocks of S alone before the others), with three places in it: dQ, dP one block ahead, S two blocks ahead. A place is a tile's number, the
        // block and the number of blocks; those of the last four tiles are kept for the places behind the first.
        struct At {
            uint32_t tile = 0;
            int j = 0, n = 0, skip = 0;
            // of a tile's entry below: its blocks, negative where it is walked twice
            __device__ __forceinline__ void begin(int blocks) {
                j = 0;
                n = ADDITIVE && blocks < 0 ? -2 * blocks : blocks;
                skip = ADDITIVE && blocks < 0 ? -blocks : 0;
            }
        };
        uint32_t k = 0, su = 0, ds = 0, dp = 0;               // ring entries, S issued, dS (or freed S) taken, dP issued
        At at_s, at_dp, at_dq;
        Place<C::kK> ka, kb;                                  // K of S, of dQ
        Place<C::kV> v;
        bool alive = true, issued = false;
        int kept0 = 0, kept1 = 0, kept2 = 0, kept3 = 0;
        auto next_work = [&]() {                              // at_s: the next tile, n = 0 behind the last
            const int e = next_tile(k++, ring, sc);
            const bool twice = ADDITIVE && e < -1;
            const int t = twice ? twice_entry(e) : e;
            int n = t < 0 ? 0 : q_tile<PARTS>(t, p).n;
            if (twice) n = -n;
            at_s.begin(n);
            const uint32_t i = at_s.tile & 3u;
            kept0 = i == 0 ? n : kept0;
            kept1 = i == 1 ? n : kept1;
            kept2 = i == 2 ? n : kept2;
            kept3 = i == 3 ? n : kept3;
        };
        auto go_on = [&](At& a) {
            if (++a.j < a.n) return;
            ++a.tile;
            const uint32_t i = a.tile & 3u;
            a.begin(i == 0 ? kept0 : i == 1 ? kept1 : i == 2 ? kept2 : kept3);
        };
        // Second halves of the products that are half issued: of S (s_open), with its buffers and what follows it, of dP, dQ
        bool s_open = false, s_ends = false, dp_open = false, dp_ends = false, dq_open = false, dq_ends = false;
        uint32_t s_tile = 0, s_buf = 0, dp_tile = 0, dq_tile = 0, dq_buf = 0;
        auto rest = [&] {
            if (s_open) {
                half_over_d<D, BF16>(1, tmem + C::cS + 128 * s_buf, smem + C::kQOff, smem + C::kKOff + s_tile * T::kBytes);
                ptx::tc_commit(bar(C::bS + s_buf));
                if (s_ends) ptx::tc_commit(bar(C::bQEmpty));
            }
            if (dp_open) {
                half_over_d<D, BF16>(1, tmem + C::cDP, smem + C::kGOff, smem + C::kVOff + dp_tile * T::kBytes);
                ptx::tc_commit(bar(C::bDP));
                ptx::tc_commit(bar(C::bVEmpty + dp_tile));
                if (dp_ends) ptx::tc_commit(bar(C::bGEmpty));
            }
            if (dq_open) {
                half_over_rows<D, BF16>(1, tmem + C::cDQ, tmem + C::cS + 128 * dq_buf, smem + C::kKOff + dq_tile * T::kBytes, true);
                ptx::tc_commit(bar(C::bKEmpty + dq_tile));
                if (dq_ends) ptx::tc_commit(bar(C::bAcc));
            }
        };
        auto close = [&] { s_open = dp_open = dq_open = false; };
        auto begin_s = [&]() -> bool {
            const uint32_t b = bar(C::bK + ka.at), par = ka.parity(), qb = bar(C::bQ), qpar = at_s.tile & 1u;
            const bool first = at_s.j == 0;
            if (!follow(
                    first ? warp_test2(b, par, qb, qpar) : warp_test(b, par),
                    [&] { return warp_wait(b, par, sc) && (!first || warp_wait(qb, qpar, sc)); }, rest,
                    [&] {
                        half_over_d<D, BF16>(0, tmem + C::cS + 128 * (su & 1u), smem + C::kQOff, smem + C::kKOff + ka.at * T::kBytes);
                    }))
                return false;
            close();
            s_open = issued = true;
            s_tile = ka.at;
            s_buf = su & 1u;
            s_ends = at_s.j + 1 == at_s.n;
            ++su;
            ka = ka.next();
            if (s_ends) {
                // the loads of a further tile wait for this product, whose end may wait for nothing then
                if (ptx::elect_one()) rest();
                close();
                ++at_s.tile;
                next_work();
            } else {
                ++at_s.j;
            }
            return true;
        };
        auto begin_dp = [&]() -> bool {
            if (!ADDITIVE || at_dp.j >= at_dp.skip) {
                const uint32_t b = bar(C::bV + v.at), par = v.parity(), fb = bar(C::bDPFree), fpar = (dp - 1) & 1u;
                const bool first = at_dp.j == at_dp.skip;
                const uint32_t gpar = at_dp.tile & 1u;
                if (!follow(
                        dp > 0 && !first && warp_test2(b, par, fb, fpar),
                        [&] {
                            return warp_wait(b, par, sc) && (dp == 0 || warp_wait(fb, fpar, sc)) &&
                                   (!first || warp_wait(bar(C::bG), gpar, sc));
                        },
                        rest,
                        [&] { half_over_d<D, BF16>(0, tmem + C::cDP, smem + C::kGOff, smem + C::kVOff + v.at * T::kBytes); }))
                    return false;
                close();
                dp_open = true;
                dp_tile = v.at;
                dp_ends = at_dp.j + 1 == at_dp.n;
                ++dp;
                v = v.next();
            }
            go_on(at_dp);
            return true;
        };
        auto begin_dq = [&]() -> bool {
            const uint32_t b = bar(C::bDS + (ds & 1u)), par = (ds >> 1) & 1u;
            if (ADDITIVE && at_dq.j < at_dq.skip) {          // S alone, which the warps have read
                if (ptx::elect_one()) rest();
                close();
                if (!warp_wait(b, par, sc)) return false;
                commit(bar(C::bKEmpty + kb.at));
            } else {
                const bool first = at_dq.j == at_dq.skip, drained = !first || at_dq.tile == 0;
                const uint32_t apar = (at_dq.tile - 1) & 1u;  // the warps have the last tile's dQ
                if (!follow(
                        drained ? warp_test(b, par) : warp_test2(b, par, bar(C::bAccEmpty), apar),
                        [&] { return warp_wait(b, par, sc) && (drained || warp_wait(bar(C::bAccEmpty), apar, sc)); }, rest,
                        [&] {
                            half_over_rows<D, BF16>(0, tmem + C::cDQ, tmem + C::cS + 128 * (ds & 1u),
                                                    smem + C::kKOff + kb.at * T::kBytes, !first);
                        }))
                    return false;
                close();
                dq_open = true;
                dq_tile = kb.at;
                dq_buf = ds & 1u;
                dq_ends = at_dq.j + 1 == at_dq.n;
            }
            ++ds;
            kb = kb.next();
            go_on(at_dq);
            return true;
        };
        if (p.stall) alive = warp_wait(bar(C::bStall), 0, sc);               // nothing ever arrives
        if (alive) {
            next_work();
            at_dp = at_dq = at_s;
            alive = at_s.n == 0 || (begin_s() && begin_dp() && (at_s.n == 0 || begin_s()));
        }
        while (alive && at_dq.n > 0)
            alive = (at_dp.n == 0 || begin_dp()) && begin_dq() && (at_s.n == 0 || begin_s());
        if (alive && ptx::elect_one()) rest();
        if (issued) {
            commit(bar(C::bDrain));
            drain_phase(bar(C::bDrain), 0, sc);
        }
        __syncwarp();
    } else if (warp < kWarps) {
        // ---------------------------------------------------------------- dS
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane;     // query of the tile; columns kCols wg ..
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + C::cS + kCols * wg, tDP = tmem + lane_base + C::cDP + kCols * wg;
        const float sl = p.scale_log2;
        int shift = 0;                                            // of the tile
        float more = 1.f, back = 1.f;                             // 2^shift; 2^-shift of the tile before
        float2* stat = reinterpret_cast<float2*>(smem_ptr + C::kStatOff);
        uint32_t tiles = 0, su = 0, dp = 0, seen = 0;
        bool alive = true;
        // Each warpgroup writes 32 columns of dQ: of the tile before, once the first block of the next one is in registers
        const bool writes = 32 * wg < D;
        void* done_row = nullptr;
        bool done_there = false;
        auto finish = [&]() -> bool {
            if (!done_row) return true;
            if (!warp_wait(bar(C::bAcc), tiles & 1u, sc)) return false;
            ptx::tc_fence_after_sync();
            if (PARTS && writes)
                store_part<32>(tmem + lane_base + C::cDQ + 32 * wg, bar(C::bAccEmpty), static_cast<float*>(done_row), back, done_there);
            else if (writes)
                store_row<32, BF16>(tmem + lane_base + C::cDQ + 32 * wg, bar(C::bAccEmpty), static_cast<uint16_t*>(done_row),
                                    p.scale * back, done_there, p.vec8);
            else
                warp_arrive(bar(C::bAccEmpty));
            done_row = nullptr;
            ++tiles;
            return true;
        };
        for (uint32_t k = 0; alive; ++k) {
            const int e = next_tile(k, ring, sc);
            const bool twice = ADDITIVE && e < -1;
            const int t = twice ? twice_entry(e) : e;
            if (t < 0) break;
            const QTile w = q_tile<PARTS>(t, p);
            const uint32_t range = range_of<BF16>(p, w.b, w.hk);
            const int row = w.m0 + r;
            const bool there = row < p.Sq;
            const size_t at = ((size_t)w.b * p.Hq + w.h) * p.Sp + row;
            // keys [low, lim) are visible, and those before sinks
            const int lim = p.causal ? min(p.Sk, max(0, row + p.off + 1)) : p.Sk;
            const int low = p.window ? row + p.off - p.window + 1 : 0;
            float nl = 0.f, is = 0.f, nd = 0.f;
            if (!twice) {
                const float l = there ? p.lse[((size_t)w.b * p.Hq + w.h) * p.Sq + row] : -INFINITY;
                const bool any = l != -INFINITY;
                nl = any ? -l * kLog2E : ADDITIVE ? 0.f : -INFINITY;
                is = any ? 1.f : 0.f;
            }
            // delta of the tile's rows, eight a warp, O from device memory (whole lines of it) and dO from its tile
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kPasses = 8 / kAtOnce;              // lanes of a row
            const int r0 = 8 * warp + lane / kLanes, piece = lane % kLanes;
            auto fetch_o = [&](uint4 (&o)[kPasses]) {
                const uint16_t* at_o = p.o + (((size_t)w.b * p.Sq + w.m0 + r0) * p.Hq + w.h) * D + 8 * piece;
#pragma unroll
                for (int e = 0; e < kPasses; ++e)
                    o[e] = w.m0 + r0 + kAtOnce * e < p.Sq
                               ? __ldcg(reinterpret_cast<const uint4*>(at_o + (size_t)(kAtOnce * e) * p.Hq * D))
                               : make_uint4(0u, 0u, 0u, 0u);
            };
            auto find_delta = [&](const uint4 (&o)[kPasses]) -> bool {
                if (!warp_wait(bar(C::bG), k & 1u, sc)) return false;
                float* delta = reinterpret_cast<float*>(smem_ptr + C::kDeltaOff);
#pragma unroll
                for (int e = 0; e < kPasses; ++e) {
                    const int i = r0 + kAtOnce * e;
                    const uint4 g = *reinterpret_cast<const uint4*>(smem_ptr + C::kGOff + (piece >> 3) * T::kBoxBytes + i * 128 +
                                                                    (((piece & 7) ^ (i & 7)) << 4));
                    const uint32_t a[4] = {o[e].x, o[e].y, o[e].z, o[e].w}, c[4] = {g.x, g.y, g.z, g.w};
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const float2 x = widen<BF16>(a[f]), y = widen<BF16>(c[f]);
                        s0 = fmaf(x.x, y.x, s0);
                        s1 = fmaf(x.y, y.y, s1);
                    }
                    s0 += s1;
#pragma unroll
                    for (int m = kLanes / 2; m > 0; m >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, m);
                    if (piece == 0) delta[i] = -s0;
                }
                warp_arrive(bar(C::bDelta));
                if (!warp_wait(bar(C::bDelta), k & 1u, sc)) return false;
                nd = delta[r];
                warp_arrive(bar(C::bGEmpty));                     // (the next tile's are written after its dO has come)
                more = power_of_two(shift);
                if (wg == 0 && w.split == 0) {
                    p.neg_delta[at] = nd * power_of_two(shift - kPShift<BF16>);
                    if (!twice) p.neg_lse[at] = ADDITIVE ? nl : nl + (float)kPShift<BF16>;
                    if (ADDITIVE && !twice) p.inv_sum[at] = is * power_of_two(kPShift<BF16>);
                }
                if (ADDITIVE) is *= more;
                else nd *= more;
                return true;
            };

            // logits in log2 units of block j: S in the buffer of `su`, scaled, masked, hidden keys at -inf
            auto logits = [&](int j, float* x) -> bool {
                const int key0 = w.block(j) * kBlock + kCols * wg;
                float m[kCols];
                if (ADDITIVE) load_mask(m, p.mask + (size_t)w.b * p.Sq * p.Sk, w.m0 + (warp & 3) * 32, p.Sq, key0, p.Sk);
                if (!warp_wait(bar(C::bS + (su & 1u)), (su >> 1) & 1u, sc)) return false;
                ptx::tc_fence_after_sync();
                if (ADDITIVE) {
                    load32(tS + 128 * (su & 1u), x);
#pragma unroll
                    for (int c = 0; c < kCols; ++c) x[c] = fmaf(m[c], kLog2E, x[c] * sl);
                } else {
                    load32(tS + 128 * (su & 1u), x);
#pragma unroll
                    for (int c = 0; c < kCols; c += 2) ptx::fma2(x[c], x[c + 1], x[c], x[c + 1], sl, sl, nl, nl);
                }
                const int c1 = lim - key0, c0 = low - key0, cs = p.sinks - key0;
                if (c1 < kCols || (p.window && c0 > 0 && cs < kCols)) {
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c >= c1 || (p.window && c < c0 && c >= cs)) x[c] = -INFINITY;
                }
                return true;
            };

            if (twice) {
                float m = -INFINITY, l = 0.f;
                for (int j = 0; j < w.n; ++j, ++su) {
                    float x[kCols];
                    if (!(alive = logits(j, x))) break;
                    warp_arrive_tmem(bar(C::bDS + (su & 1u)));
                    if (j == 0 && !(alive = finish())) break;
                    float top = m;
#pragma unroll
                    for (int c = 0; c < kCols; c += 2) top = ptx::max3(top, x[c], x[c + 1]);
                    if (top != -INFINITY) {
                        l *= ptx::ex2(m - top);
                        m = top;
#pragma unroll
                        for (int c = 0; c < kCols; ++c) l += ptx::ex2(x[c] - top);
                    }
                }
                if (!alive) break;
                // the first warpgroup joins the parts of the row
                if (wg) {
                    stat[128 * wg + r] = make_float2(m, l);
                    warp_arrive(bar(C::bParts));
                    if (!(alive = warp_wait(bar(C::bWhole), seen & 1u, sc))) break;
                } else {
                    if (!(alive = warp_wait(bar(C::bParts), seen & 1u, sc))) break;
#pragma unroll
                    for (int g = 1; g < kGroups; ++g) {
                        const float2 o = stat[128 * g + r];
                        const float top = fmaxf(m, o.x);
                        if (top != -INFINITY) l = l * ptx::ex2(m - top) + o.y * ptx::ex2(o.x - top);
                        m = top;
                    }
                    const bool any = there && l > 0.f;
                    stat[r] = make_float2(any ? -m : 0.f, any ? 1.f / l : 0.f);
                    p.neg_lse[at] = stat[r].x;
                    p.inv_sum[at] = stat[r].y * power_of_two(kPShift<BF16>);
                    warp_arrive(bar(C::bWhole));
                }
                ++seen;
                nl = stat[r].x;
                is = stat[r].y;
            }
            // The first block of a tile is a copy of its own: it has the last tile's dQ and delta to see to.
            auto block = [&](int j, auto begins) -> bool {
                float x[kCols];
                uint4 o[kPasses];
                if constexpr (decltype(begins)::value) fetch_o(o);
                if (!logits(j, x)) return false;
                if constexpr (decltype(begins)::value) shift = ds_shift<BF16>(range);
#pragma unroll
                for (int c = 0; c < kCols; ++c) x[c] = ptx::ex2(ADDITIVE ? x[c] + nl : x[c]);
                if constexpr (decltype(begins)::value) {
                    if (!finish()) return false;
                    if (!find_delta(o)) return false;
                }
                if (!warp_wait(bar(C::bDP), dp & 1u, sc)) return false;
                ptx::tc_fence_after_sync();
                float d[kCols];
                uint32_t pk[kCols / 2];
                load32(tDP, d);
                warp_arrive_tmem(bar(C::bDPFree));
#pragma unroll
                for (int c = 0; c < kCols; c += 2) {
                    if (BF16 || ADDITIVE) ptx::add2(d[c], d[c + 1], d[c], d[c + 1], nd, nd);
                    else ptx::fma2(d[c], d[c + 1], d[c], d[c + 1], more, more, nd, nd);
                    if (ADDITIVE) ptx::mul2(d[c], d[c + 1], d[c], d[c + 1], is, is);
                    ptx::mul2(d[c], d[c + 1], d[c], d[c + 1], x[c], x[c + 1]);
                    pk[c / 2] = pack<BF16>(d[c], d[c + 1]);
                }
                ptx::tmem_st16(tS + 128 * (su & 1u), pk);
                ptx::tmem_st_wait();
                warp_arrive_tmem(bar(C::bDS + (su & 1u)));
                ++su;
                ++dp;
                return true;
            };
            alive = block(0, std::true_type{});
            for (int j = 1; j < w.n && alive; ++j) alive = block(j, std::false_type{});
            if (!alive) break;
            const long long token = (long long)w.b * p.Sq + row;
            void* out = static_cast<uint16_t*>(p.dq) + token * p.dq_stride + w.h * D + 32 * wg;
            if (PARTS)
                out = p.part + w.split * ((long long)p.B * p.Sq * p.Hq * D) + (token * p.Hq + w.h) * D + 32 * wg;
            done_row = out;
            done_there = there;
            back = power_of_two(-shift);
        }
        if (alive) finish();
    }

    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kIssueWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace bwd
}  // namespace attn
