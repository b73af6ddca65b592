// Appending a step's keys and values to a paged cache, the keys rotated to
// their positions on the way, and quantised when the cache holds 8 bits.
//
// Token s of sequence b sits at position pos = kv_lens[b] - new_lens[b] + s:
// page block_table[b][pos / page], slot pos % page. A page of one K/V head is
// one contiguous (page, D) block of the cache and, in an 8-bit cache, has one
// scale for its keys and one for its values. One CTA owns one such block: it
// alone reads and writes the block's scale and slots, so nothing is atomic and
// results do not depend on the order of the CTAs.
//
// 8-bit blocks hold e4m3 codes and a power-of-two scale 2^e, the smallest with
// max |x| <= 448 * 2^e over the block's values. A block whose scale grows
// under new tokens has its earlier codes multiplied by 2^(old - new), which
// moves their exponents and is exact except where a code enters the subnormal
// range (below 2^-6 * scale); an arbitrary scale would round every code again
// each time. e4m3 has the same relative precision under any scale, so the
// power of two costs nothing else.
#include <algorithm>
#include <type_traits>

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "paged_params.h"

namespace attn {
namespace paged {
namespace {

// A block's new tokens as 16-byte pieces (eight values): HELD a thread. Steps of
// few tokens have one piece a thread and up to 512 threads, prompts four and up
// to 256, large pages eight and up to 512 (256 tokens of 16 pieces). (4 x 2048
// tokens, 32 heads of 128 into e4m3 pages of 16, 64, 128, 256: 65.6, 41.0, 47.6, 68.2
// us; over e4m3 four pieces spill 24 bytes a thread, eight 92 to 120.)
__host__ __device__ constexpr int max_threads(int held) { return held == 4 ? 256 : 512; }
__host__ __device__ constexpr int min_ctas(int held) { return held == 4 ? 3 : 1; }

// Four floats to four e4m3 codes (round to nearest even, beyond +-448 to
// +-448, NaN stays NaN), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
    uint32_t h;
    float2 f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
    float2 f;
    if (BF16) {
        f.x = __uint_as_float(w << 16);
        f.y = __uint_as_float(w & 0xffff0000u);
    } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(f.x), "=f"(f.y)
            : "r"(w));
    }
    return f;
}

// The smallest 2^e >= 2^kMinScaleExp with a <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float block_scale(float a) {
    const uint32_t bits = __float_as_uint(a);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, kMinScaleExp);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// One CTA per (sequence, touched page, group of K/V heads, keys or values); it
// takes the blocks of its heads one after the other, every thread holding the
// same slots and dims of each, so that a page's table entries come from L1
// after the first head. A block's new values stay in registers (FP32, rotated)
// between the pass that finds their maximum and the one that writes them.
// Bound by memory: each input is read and each code written once. Measured: 4 x
// 2048 tokens of 32 heads of 128 into e4m3 pages of 64 (bf16, rotated) 41 us,
// 5.0 TB/s of the 6.70 a copy reaches; the conversions and the block's maximum
// stand between a block's loads and its stores, and the next block's loads
// overlap only in part (staging them by asynchronous copies: 43 to 47 us). Few
// tokens are bound by latency: one token of 64 sequences 2.4 us, 8 x 500 tokens
// into 16-bit pages 4.1 us.
template <bool E4M3, int HELD, bool BF16>
__global__ void __launch_bounds__(max_threads(HELD), min_ctas(HELD)) append_kernel(const AppendParams p) {
    __shared__ float red[2][max_threads(HELD) / 32];
    wait_for_inputs();
    let_next_start();
    const int is_v = blockIdx.x & 1;
    long long u = blockIdx.x >> 1;
    const int groups = (p.Hkv + p.head_group - 1) / p.head_group;
    const int h0 = (int)(u % groups) * p.head_group, h1 = min(p.Hkv, h0 + p.head_group);
    u /= groups;
    const int j = (int)(u % p.touched);
    const int b = (int)(u / p.touched);
    const int page = 1 << p.page_shift;

    const int kv = p.kv_lens[b], n_new = p.new_lens ? p.new_lens[b] : p.S;
    if (n_new == 0) return;
    // Lengths the table or the step cannot hold: nothing of the sequence is written.
    if (n_new < 0 || n_new > p.S || kv < n_new || (kv - 1) >> p.page_shift >= p.max_pages ||
        (p.rope && kv > p.max_pos)) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
        return;
    }
    const int first = kv - n_new;                      // position of the step's first token
    const int pg = (first >> p.page_shift) + j;
    if (pg > (kv - 1) >> p.page_shift) return;
    const int id = p.block_table[(size_t)b * p.max_pages + pg];
    if ((unsigned)id >= (unsigned)p.n_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
        return;
    }
    const int pos0 = max(first, pg << p.page_shift);   // the page's first new token, and one past its last
    const int pos1 = min(kv, (pg + 1) << p.page_shift);
    const int slot0 = pos0 & (page - 1);
    const int chunks = p.D / 8, cshift = p.D == 128 ? 4 : 3;   // pieces of a token
    const int n = (pos1 - pos0) * chunks;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    const uint16_t* const src = (is_v ? p.v : p.k) + ((long long)b * p.S + (pos0 - first)) * stride;
    const bool turn = !is_v && p.rope != nullptr;
    const float4* const table = reinterpret_cast<const float4*>(p.rope) + (size_t)pos0 * (p.D / 4);

    // A thread's pieces are whole tokens apart (the threads are a multiple of a
    // token's pieces). Raw pieces of the next head are fetched while the current
    // one is worked on.
    const uint16_t* const src_t = src + (threadIdx.x >> cshift) * stride + 8 * (threadIdx.x & (chunks - 1));
    const long long apart = (blockDim.x >> cshift) * stride;
    auto there = [&](int c) { return c < n; };
    uint4 w[HELD];
    auto fetch = [&](int h) {
        const uint16_t* const at = src_t + h * p.D;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (there(c)) w[i] = __ldcg(reinterpret_cast<const uint4*>(at + i * apart));
        }
    };
    fetch(h0);
    for (int h = h0; h < h1; ++h) {
        const size_t block = ((size_t)id * p.Hkv + h) << p.page_shift;
        float* const scale_at = E4M3 ? (is_v ? p.v_scale : p.k_scale) + (size_t)id * p.Hkv + h : nullptr;
        const float before = E4M3 && slot0 > 0 ? *scale_at : 0.f;
        float x[HELD][8];
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = widen<BF16>(ws[e]);
                x[i][2 * e] = f.x;
                x[i][2 * e + 1] = f.y;
            }
            if (turn && there(c)) {
                const float4 a0 = __ldg(table + 2 * c), a1 = __ldg(table + 2 * c + 1);
                const float cs[4] = {a0.x, a0.z, a1.x, a1.z}, sn[4] = {a0.y, a0.w, a1.y, a1.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f0 = x[i][2 * e], f1 = x[i][2 * e + 1];
                    x[i][2 * e] = f0 * cs[e] - f1 * sn[e];
                    x[i][2 * e + 1] = f1 * cs[e] + f0 * sn[e];
                }
            }
        }
        if (h + 1 < h1) fetch(h + 1);
        if (!E4M3) {
            uint4* const dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) +
                                                        (block + slot0) * p.D);
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                uint32_t r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r[e] = BF16 ? ptx::pack_bf16x2(x[i][2 * e], x[i][2 * e + 1])
                                  : ptx::pack_f16x2(x[i][2 * e], x[i][2 * e + 1]);
                if (there(c)) dst[c] = make_uint4(r[0], r[1], r[2], r[3]);
            }
            continue;
        }

        float a = 0.f;
#pragma unroll
        for (int i = 0; i < HELD; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[i][e]));      // (passes NaN over)
        if (a > 3.402823466e38f) {                     // infinities do not set the scale
            a = 0.f;
#pragma unroll
            for (int i = 0; i < HELD; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[i][e]) <= 3.402823466e38f ? fabsf(x[i][e]) : 0.f);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        float* const r2 = red[(h - h0) & 1];           // two in turn: one barrier a head
        if ((threadIdx.x & 31) == 0) r2[threadIdx.x >> 5] = a;
        __syncthreads();
        for (int w = 0; w < (int)blockDim.x / 32; ++w) a = fmaxf(a, r2[w]);

        uint8_t* const blk = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + block * p.D;
        float scale = block_scale(a);
        if (slot0 > 0) {
            // Earlier tokens share the block: its scale only grows, and their codes move with it.
            scale = fmaxf(before, scale);
            if (scale != before) {
                const float f = before / scale;
                uint2* old = reinterpret_cast<uint2*>(blk);
                for (int c = threadIdx.x; c < slot0 * chunks; c += blockDim.x) {
                    const uint2 w = old[c];
                    const uint32_t ws[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
                    float2 v2[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v2[i] = from_e4m3x2(ws[i]);
                    old[c] = make_uint2(to_e4m3x4(v2[0].x * f, v2[0].y * f, v2[1].x * f, v2[1].y * f),
                                        to_e4m3x4(v2[2].x * f, v2[2].y * f, v2[3].x * f, v2[3].y * f));
                }
            }
        }
        if (threadIdx.x == 0) *scale_at = scale;       // every thread read the old one before the barrier
        const float inv = 1.f / scale;                 // exact: a power of two in range
        uint2* const dst = reinterpret_cast<uint2*>(blk + (size_t)slot0 * p.D);
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
            for (int e = 0; e < 8; e += 2) ptx::mul2(x[i][e], x[i][e + 1], x[i][e], x[i][e + 1], inv, inv);
            if (there(c))
                dst[c] = make_uint2(to_e4m3x4(x[i][0], x[i][1], x[i][2], x[i][3]),
                                    to_e4m3x4(x[i][4], x[i][5], x[i][6], x[i][7]));
        }
    }
}

}  // namespace

int launch_append(AppendParams p, int cache, int num_sms, cudaStream_t stream) {
    // Heads a CTA takes in turn: table entries are read once per group, but only
    // where the blocks fill the SMs several times over without it. (4 x 2048
    // tokens, 32 heads into e4m3: 1, 2, 3, 4 heads 56, 44.7, 41.9, 40.8 us.)
    const long long blocks = (long long)p.B * p.touched * p.Hkv * 2;
    p.head_group = (int)std::max(1LL, std::min<long long>(std::min(p.Hkv, 4), blocks / (8LL * num_sms)));
    const int groups = (p.Hkv + p.head_group - 1) / p.head_group;
    const unsigned grid = (unsigned)((long long)p.B * p.touched * groups * 2);
    const int pieces = std::min(p.S, 1 << p.page_shift) * (p.D / 8);
    auto run = [&](auto kernel, int held) {
        const int threads = ((pieces + held - 1) / held + 31) / 32 * 32;
        if (launch_early(kernel, grid, threads, 0, stream, p) != cudaSuccess) return ATTN_ERR_CUDA;
        return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    };
    auto pick = [&](auto e4m3, auto bf16) {
        constexpr bool kE = decltype(e4m3)::value, kB = decltype(bf16)::value;
        if (pieces <= max_threads(1)) return run(append_kernel<kE, 1, kB>, 1);
        return pieces <= 4 * max_threads(4) ? run(append_kernel<kE, 4, kB>, 4) : run(append_kernel<kE, 8, kB>, 8);
    };
    if (cache == kE4m3)
        return p.bf16 ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
    return p.bf16 ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
}

}  // namespace paged
}  // namespace attn
