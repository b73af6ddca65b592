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
#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "paged_params.h"

namespace attn {
namespace paged {
namespace {

constexpr int kThreads = 128;

// Two floats to two e4m3 codes (round to nearest even, beyond +-448 to +-448,
// NaN stays NaN); `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
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

__device__ __forceinline__ float2 widen(uint32_t w, bool bf16) {
    float2 f;
    if (bf16) {
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

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) v = fmaxf(v, red[w]);
    return v;
}

// One CTA per (sequence, touched page, K/V head, keys or values).
template <bool E4M3>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    __shared__ float red[kThreads / 32];
    const int is_v = blockIdx.x & 1;
    long long u = blockIdx.x >> 1;
    const int h = (int)(u % p.Hkv);
    u /= p.Hkv;
    const int j = (int)(u % p.touched);
    const int b = (int)(u / p.touched);
    const int page = 1 << p.page_shift;

    int kv = p.kv_lens[b], n_new = p.new_lens ? p.new_lens[b] : p.S;
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
    const int chunks = p.D / 8;                        // 16-byte pieces (eight values) of a token
    const int n = (pos1 - pos0) * chunks;
    const uint16_t* src = (is_v ? p.v : p.k) + ((long long)b * p.S + (pos0 - first)) * (is_v ? p.v_stride : p.k_stride) +
                          (long long)h * p.D;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    const bool turn = !is_v && p.rope != nullptr;
    const size_t block = ((size_t)id * p.Hkv + h) << p.page_shift;

    auto load = [&](int c, float* x) {
        const int t = c / chunks, g = c - t * chunks;
        const uint4 w = *reinterpret_cast<const uint4*>(src + t * stride + 8 * g);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        float4 a0 = make_float4(1.f, 0.f, 1.f, 0.f), a1 = a0;
        if (turn) {
            const float4* at = reinterpret_cast<const float4*>(p.rope) + (size_t)(pos0 + t) * (p.D / 4) + 2 * g;
            a0 = __ldg(at);
            a1 = __ldg(at + 1);
        }
        const float cs[4] = {a0.x, a0.z, a1.x, a1.z}, sn[4] = {a0.y, a0.w, a1.y, a1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen(ws[i], p.bf16);
            x[2 * i] = turn ? f.x * cs[i] - f.y * sn[i] : f.x;
            x[2 * i + 1] = turn ? f.y * cs[i] + f.x * sn[i] : f.y;
        }
    };

    if (!E4M3) {
        uint16_t* dst = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + (block + slot0) * p.D;
        for (int c = threadIdx.x; c < n; c += kThreads) {
            float x[8];
            load(c, x);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = p.bf16 ? ptx::pack_bf16x2(x[2 * i], x[2 * i + 1]) : ptx::pack_f16x2(x[2 * i], x[2 * i + 1]);
            *reinterpret_cast<uint4*>(dst + 8 * (size_t)c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return;
    }

    float a = 0.f;
    for (int c = threadIdx.x; c < n; c += kThreads) {
        float x[8];
        load(c, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float m = fabsf(x[i]);
            a = fmaxf(a, m <= 3.402823466e38f ? m : 0.f);        // NaN and infinities do not set the scale
        }
    }
    a = block_max(a, red);
    uint8_t* blk = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + block * p.D;
    float* scale_at = (is_v ? p.v_scale : p.k_scale) + (size_t)id * p.Hkv + h;
    float scale = block_scale(a);
    if (slot0 > 0) {
        // Earlier tokens share the block: its scale only grows, and their codes move with it.
        const float before = *scale_at;
        scale = fmaxf(before, scale);
        if (scale != before) {
            const float f = before / scale;
            uint2* old = reinterpret_cast<uint2*>(blk);
            for (int c = threadIdx.x; c < slot0 * chunks; c += kThreads) {
                uint2 w = old[c];
                const uint32_t ws[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
                uint32_t r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v2 = from_e4m3x2(ws[i]);
                    r[i] = to_e4m3x2(v2.x * f, v2.y * f);
                }
                old[c] = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
            }
        }
    }
    __syncthreads();                                   // every thread has read the old scale
    if (threadIdx.x == 0) *scale_at = scale;
    const float inv = 1.f / scale;                     // exact: a power of two in range
    uint2* dst = reinterpret_cast<uint2*>(blk + (size_t)slot0 * p.D);
    for (int c = threadIdx.x; c < n; c += kThreads) {
        float x[8];
        load(c, x);
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = to_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
        dst[c] = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
    }
}

}  // namespace

int launch_append(const AppendParams& p, int cache, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const unsigned grid = (unsigned)((long long)p.B * p.touched * p.Hkv * 2);
    if (cache == kE4m3)
        append_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else
        append_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace paged
}  // namespace attn
