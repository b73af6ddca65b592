// Activation checkpoints in 8 bits: e4m3 codes of a (B, S, H, D) tensor and one
// scale 2^e for each of its head vectors, the smallest (>= 2^-100) with
// max |x| <= 448 * 2^e. A power of two moves exponents alone, so a value loses
// bits in the code and nowhere else (half a step of four significant bits, or
// 2^-10 of the scale where the code is subnormal), and the way back is exact in
// bf16. Infinities become +-448 codes and NaN stays NaN; neither sets the scale.
//
// Both directions are bound by memory: 16 bits a value on one side, 8 on the
// other, 4 bytes a vector. A vector lies in D / 16 neighbouring lanes, 16 values
// each, so that its maximum takes two or three shuffles; a lane has kVectors of
// them in flight: two, since at these sizes the first loads and the last stores are
// a good part of a launch, and small blocks even them out. Measured, 4 x 2048 tokens
// of 32 heads of 128: stored out of a packed projection in 18.1 us, 5.6 TB/s (84% of a
// copy; with four in flight 20.2, with one 19.1), loaded in 19.3 (21.3 with four, 23.2 with eight).
#include <algorithm>

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "checkpoint_params.h"
#include "e4m3.cuh"

namespace attn {
namespace checkpoint {
namespace {

constexpr int kVectors = 2;

// Eight codes times a scale, in 16 bits, saturating: the code of a value near the type's largest may lie above it.
template <bool BF16>
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi, float scale) {
    const uint32_t pairs[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = from_e4m3x2(pairs[i]);
        if (BF16)
            asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(f.y * scale), "f"(f.x * scale));
        else
            asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(f.y * scale), "f"(f.x * scale));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Element of x where vector v begins. (Offsets past 32 bits cost a 64-bit division.)
__device__ __forceinline__ long long begin_of(const Tensor& t, long long v, int D) {
    if (t.stride == (long long)t.H * D) return v * D;
    const long long token = v <= 0x7fffffff ? (long long)((unsigned)v / (unsigned)t.H) : v / t.H;
    return token * t.stride + (v - token * t.H) * D;
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) store_kernel(const Tensor t) {
    wait_for_inputs();
    let_next_start();
    constexpr int kLanes = D / 16;
    const int lane = threadIdx.x % kLanes;
    const long long vectors = t.tokens * t.H;
    const long long groups = (long long)gridDim.x * (256 / kLanes);
    const long long first = (long long)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    // (whole warps stay in the loop: its bound is a warp's first group)
    for (long long v0 = first; v0 - threadIdx.x % 32 / kLanes < vectors; v0 += groups * kVectors) {
        uint4 w[kVectors][2];
#pragma unroll
        for (int u = 0; u < kVectors; ++u) {
            const long long v = v0 + u * groups;
            w[u][0] = w[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (v < vectors) {
                const uint4* src = reinterpret_cast<const uint4*>(t.x + begin_of(t, v, D)) + 2 * lane;
                w[u][0] = __ldcg(src);
                w[u][1] = __ldcg(src + 1);
            }
        }
#pragma unroll
        for (int u = 0; u < kVectors; ++u) {
            const long long v = v0 + u * groups;
            const uint32_t ws[8] = {w[u][0].x, w[u][0].y, w[u][0].z, w[u][0].w, w[u][1].x, w[u][1].y, w[u][1].z, w[u][1].w};
            float2 f[8];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = widen<BF16>(ws[i]);
                top = ptx::max3(top, finite_abs(f[i].x), finite_abs(f[i].y));
            }
#pragma unroll
            for (int m = kLanes / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
            if (v < vectors) {
                const float scale = block_scale(top);
                const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));         // 1 / 2^e
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    c[i] = to_e4m3x4(f[2 * i].x * inv, f[2 * i].y * inv, f[2 * i + 1].x * inv, f[2 * i + 1].y * inv);
                reinterpret_cast<uint4*>(t.codes)[v * kLanes + lane] = make_uint4(c[0], c[1], c[2], c[3]);
                if (lane == 0) t.scale[v] = scale;
            }
        }
    }
}

// Up to three tensors in one launch: the first `blocks[0]` blocks take the first one, and so on.
struct Tensors {
    Tensor t[3];
    int blocks[3];
};

template <int D, bool BF16>
__global__ void __launch_bounds__(256) load_kernel(const __grid_constant__ Tensors p) {
    wait_for_inputs();
    let_next_start();
    constexpr int kLanes = D / 16;
    const int b1 = p.blocks[0], b2 = p.blocks[0] + p.blocks[1];
    const int which = (int)blockIdx.x < b1 ? 0 : (int)blockIdx.x < b2 ? 1 : 2;
    const Tensor& t = p.t[which];
    const long long block = (int)blockIdx.x - (which == 0 ? 0 : which == 1 ? b1 : b2);
    const int n_blocks = p.blocks[which];
    const int lane = threadIdx.x % kLanes;
    const long long vectors = t.tokens * t.H;
    const long long groups = (long long)n_blocks * (256 / kLanes);
    for (long long v0 = block * (256 / kLanes) + threadIdx.x / kLanes; v0 < vectors; v0 += groups * kVectors) {
        uint4 w[kVectors];
        float scale[kVectors];
#pragma unroll
        for (int u = 0; u < kVectors; ++u) {
            const long long v = v0 + u * groups;
            if (v < vectors) {
                w[u] = __ldcg(reinterpret_cast<const uint4*>(t.codes) + v * kLanes + lane);
                scale[u] = __ldcg(t.scale + v);
            }
        }
#pragma unroll
        for (int u = 0; u < kVectors; ++u) {
            const long long v = v0 + u * groups;
            if (v >= vectors) break;
            uint4* dst = reinterpret_cast<uint4*>(t.x + begin_of(t, v, D)) + 2 * lane;
            dst[0] = widen8<BF16>(w[u].x, w[u].y, scale[u]);
            dst[1] = widen8<BF16>(w[u].z, w[u].w, scale[u]);
        }
    }
}

template <typename F>
int for_type(int D, bool bf16, F f) {
    if (D == 128) return bf16 ? f(std::integral_constant<int, 128>{}, std::true_type{}) : f(std::integral_constant<int, 128>{}, std::false_type{});
    return bf16 ? f(std::integral_constant<int, 64>{}, std::true_type{}) : f(std::integral_constant<int, 64>{}, std::false_type{});
}

int blocks_for(const Tensor& t, int D, int most) {
    const long long per = 256 / (D / 16) * kVectors;
    return (int)std::min<long long>((t.tokens * t.H + per - 1) / per, most);
}

}  // namespace

int launch_store(const Tensor& t, int D, bool bf16, int num_sms, cudaStream_t stream) {
    return for_type(D, bf16, [&](auto d, auto b) {
        return launch_early(store_kernel<decltype(d)::value, decltype(b)::value>, (unsigned)std::max(1, blocks_for(t, D, 32 * num_sms)),
                            256u, (size_t)0, stream, t) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    });
}

int launch_load(const Tensor* t, int n, int D, bool bf16, int num_sms, cudaStream_t stream) {
    Tensors p{};
    for (int i = 0; i < n && i < 3; ++i) {
        p.t[i] = t[i];
        p.blocks[i] = blocks_for(t[i], D, 32 * num_sms);
    }
    return for_type(D, bf16, [&](auto d, auto b) {
        return launch_early(load_kernel<decltype(d)::value, decltype(b)::value>, (unsigned)(p.blocks[0] + p.blocks[1] + p.blocks[2]),
                            256u, (size_t)0, stream, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    });
}

}  // namespace checkpoint
}  // namespace attn
