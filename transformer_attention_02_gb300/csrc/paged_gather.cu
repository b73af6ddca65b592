// Long chunks of queries over a paged cache: the pages that the queries see are
// gathered into contiguous 16-bit tensors, with the queries rotated beside
// them, and the fused tcgen05 kernel (its ragged variants) reads those.
//
// From kChunkRows queries a sequence the products outweigh the cache's reads,
// and they belong on tcgen05: the kernel of paged_attn.cuh reaches some 330
// TFLOP/s there (mma.sync, the cache read once per 32 rows), this path the
// fused kernel's rate less one pass over the cache: 16 x 256 queries over 8192
// e4m3 keys (32/8 heads of 128) 566 us, 956 TFLOP/s; one chunk of 2048 over 16384
// 428 us, 1204 TFLOP/s. Keys and values become
// code * scale, exact in bf16 for power-of-two scales (four significant bits).
// Bound by memory: each visible page is read once and written once at 16 bits.
#include <type_traits>

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "paged_params.h"

namespace attn {
namespace paged {
namespace {

constexpr int kThreads = 256;

// Eight values as they stand in the cache.
template <int CT>
using Raw = std::conditional_t<CT == kE4m3, uint2, uint4>;

// code * scale in 16 bits, saturating: the code of a value near the type's
// largest may lie above it.
__device__ __forceinline__ uint4 widen_piece(uint2 w, float scale, bool bf16) {
    const uint16_t pairs[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        float lo, hi;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pairs[i]));
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        lo *= scale, hi *= scale;
        if (bf16)
            asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(hi), "f"(lo));
        else
            asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(hi), "f"(lo));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ uint4 widen_piece(uint4 w, float, bool) { return w; }

// CTAs [0, p.copies): 128 keys of one K/V head of a sequence, zeros for those that
// no query sees, past its last key (the products read whole blocks of 128) and in
// pages out of range (which the products' kernel hides: it has the table). The
// others: 16-byte pieces of the queries, rotated to their positions. 8-bit pages in
// five CTAs an SM, 48 registers (four: 16 x 256 queries over 8192 keys 573 us, five 568).
template <int CT>
__global__ void __launch_bounds__(kThreads, CT == kE4m3 ? 5 : 4) gather_kernel(const GatherParams p) {
    wait_for_inputs();
    let_next_start();
    const int chunks = p.D / 8, cshift = p.D == 128 ? 4 : 3;
    if ((long long)blockIdx.x >= p.copies) {
        const long long n = (long long)p.B * p.Sq * p.Hq * chunks;
        const long long e = ((long long)blockIdx.x - p.copies) * kThreads + threadIdx.x;
        if (e >= n) return;
        const int g = (int)(e & (chunks - 1));
        const long long row = e >> cshift;                        // (b * Sq + i) * Hq + h
        const long long token = row / p.Hq;
        const int h = (int)(row - token * p.Hq), b = (int)(token / p.Sq), i = (int)(token - (long long)b * p.Sq);
        const int kv = min(max(p.kv_lens[b], 0), p.cap), ql = p.q_lens ? min(max(p.q_lens[b], 0), p.Sq) : p.Sq;
        if (i >= ql) return;
        int pos = kv - ql + i;
        if (pos >= p.max_pos) {
            if (g == 0) atomicOr(p.status, kStatusBadIndex);
            pos = p.max_pos - 1;
        }
        const uint4 w = *reinterpret_cast<const uint4*>(p.q + token * p.q_stride + (long long)h * p.D + 8 * g);
        const float4* at = reinterpret_cast<const float4*>(p.rope) + (size_t)max(pos, 0) * (p.D / 4) + 2 * g;
        const float4 a = __ldg(at), c = __ldg(at + 1);
        uint4 r;
        if (p.bf16)
            r = make_uint4(rotate_pair<true>(w.x, a.x, a.y), rotate_pair<true>(w.y, a.z, a.w),
                           rotate_pair<true>(w.z, c.x, c.y), rotate_pair<true>(w.w, c.z, c.w));
        else
            r = make_uint4(rotate_pair<false>(w.x, a.x, a.y), rotate_pair<false>(w.y, a.z, a.w),
                           rotate_pair<false>(w.z, c.x, c.y), rotate_pair<false>(w.w, c.z, c.w));
        reinterpret_cast<uint4*>(p.q_out)[e] = r;
        return;
    }
    long long u = blockIdx.x;
    const int hk = (int)(u % p.Hkv);
    u /= p.Hkv;
    const int blocks = (p.cap + 127) / 128, kb = (int)(u % blocks), b = (int)(u / blocks);
    const int raw_kv = p.kv_lens[b], raw_ql = p.q_lens ? p.q_lens[b] : p.Sq;
    if (kb == 0 && hk == 0 && threadIdx.x == 0 && (raw_kv < 0 || raw_kv > p.cap || raw_ql < 0 || raw_ql > p.Sq))
        atomicOr(p.status, kStatusBadIndex);
    const int kv = min(max(raw_kv, 0), p.cap), ql = min(max(raw_ql, 0), p.Sq);
    if (kb * 128 >= kv || ql == 0) return;
    // Oldest key of the first query's window: the sinks and the keys from it on are
    // seen by some query. Of the others whole blocks are left out, and in a block
    // with both they become zeros, whatever the cache or the table holds there: the
    // products take their values too, with weights of zero.
    const int low = p.window > 0 ? max(0, kv - ql - p.window + 1) : 0;
    if ((kb + 1) * 128 <= low && kb * 128 >= p.sinks) return;
    // kBatch pieces a thread are loaded before any is stored.
    constexpr int kBatch = 4;
    static_assert(128 * 8 % (kThreads * kBatch) == 0, "whole batches");
    for (int c0 = threadIdx.x; c0 < 128 << cshift; c0 += kBatch * kThreads) {
        Raw<CT> k[kBatch], v[kBatch];
        float ks[kBatch], vs[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int c = c0 + i * kThreads, key = kb * 128 + (c >> cshift), g = c & (chunks - 1);
            k[i] = v[i] = Raw<CT>{};
            ks[i] = vs[i] = 1.f;
            if (key < kv && (key >= low || key < p.sinks)) {
                const int id = p.block_table[(size_t)b * p.max_pages + (key >> p.page_shift)];
                if ((unsigned)id < (unsigned)p.n_pages) {
                    const size_t block = (size_t)id * p.Hkv + hk;
                    const size_t at = ((block << p.page_shift) + (size_t)(key & ((1 << p.page_shift) - 1))) * chunks + g;
                    k[i] = __ldcg(static_cast<const Raw<CT>*>(p.k_cache) + at);
                    v[i] = __ldcg(static_cast<const Raw<CT>*>(p.v_cache) + at);
                    if (CT == kE4m3) {
                        ks[i] = __ldcg(p.k_scale + block);
                        vs[i] = __ldcg(p.v_scale + block);
                    }
                } else {
                    atomicOr(p.status, kStatusBadIndex);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int c = c0 + i * kThreads, key = kb * 128 + (c >> cshift), g = c & (chunks - 1);
            if (key < p.cap) {                                    // (the tensor's end: loads past it read zeros)
                const size_t to = (((size_t)b * p.cap + key) * p.Hkv + hk) * chunks + g;
                reinterpret_cast<uint4*>(p.k_out)[to] = widen_piece(k[i], ks[i], p.bf16);
                reinterpret_cast<uint4*>(p.v_out)[to] = widen_piece(v[i], vs[i], p.bf16);
            }
        }
    }
}

}  // namespace

int launch_gather(GatherParams p, int cache, cudaStream_t stream) {
    p.copies = (long long)p.B * ((p.cap + 127) / 128) * p.Hkv;
    const long long pieces = p.rope ? (long long)p.B * p.Sq * p.Hq * (p.D / 8) : 0;
    const unsigned grid = (unsigned)(p.copies + (pieces + kThreads - 1) / kThreads);
    auto kernel = cache == kE4m3 ? gather_kernel<kE4m3> : gather_kernel<kBf16>;
    if (launch_early(kernel, grid, kThreads, 0, stream, p) != cudaSuccess) return ATTN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace paged
}  // namespace attn
