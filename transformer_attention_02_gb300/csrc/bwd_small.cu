// The small kernels around the products of the attention's backward pass: before
// them the two counters are set from which their CTAs take work tiles, and in fp16
// the largest norms of dO and V are found, which bound dS; behind them, where few tiles were
// cut into parts, the parts' FP32 sums are joined, in the parts' order.
#include <algorithm>

#include "../../include/attn.h"
#include "bwd_params.h"
#include "e4m3.cuh"
#include "early_launch.h"
#include "ptx.cuh"

namespace attn {
namespace bwd {
namespace {

__global__ void bwd_begin_kernel(unsigned int* counters) {
    wait_for_inputs();
    let_next_start();
    if (threadIdx.x < 2) counters[threadIdx.x] = 0u;
}

// Sum of the squares of eight values, infinities and NaN left out.
__device__ __forceinline__ float squares(const uint4& w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = widen<false>(x[i]);
        s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
    }
    if (!(s < INFINITY)) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen<false>(x[i]);
            s += (fabsf(f.x) < INFINITY ? f.x * f.x : 0.f) + (fabsf(f.y) < INFINITY ? f.y * f.y : 0.f);
        }
    }
    return s;
}

// A block takes a part of the head vectors of 2^shift neighbouring K/V heads, dO's and then V's, D / 8 lanes a vector. Bound by
// memory, which wants whole stretches of a token: with a head a block 4 x 2048 tokens of 32 heads of 128 take 38 us, with eight
// 32, and 27 (134 MB, 5.0 TB/s) since infinities are looked for only where a sum has met one. At small sizes bound by one wave's
// latency: four vectors in flight.
template <int D>
__global__ void __launch_bounds__(kRangeThreads, 2) bwd_range_kernel(const RangeParams p) {
    wait_for_inputs();
    let_next_start();
    constexpr int kLanes = D / 8, kVectors = kRangeThreads / kLanes;
    __shared__ float2 part[kVectors];
    if (blockIdx.x == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0u;
    const int lane = threadIdx.x % 32, piece = threadIdx.x % kLanes, vector = threadIdx.x / kLanes, heads = 1 << p.shift;
    const int per_row = p.Hkv >> p.shift;                         // units of a token
    const long long q_rows = (long long)p.Sq * p.group, rows = q_rows + p.Sk;
    const long long step = (long long)p.parts * (kVectors >> p.shift);
    for (unsigned u = blockIdx.x; u < (unsigned)p.units; u += gridDim.x) {
        const int at_heads = (int)(u / (unsigned)p.parts), split = (int)u - at_heads * p.parts, b = at_heads / per_row;
        const int hk = ((at_heads - b * per_row) << p.shift) + (vector & (heads - 1));
        const uint16_t* const d_o = p.d_o + ((long long)b * p.Sq * p.Hkv + hk) * p.group * D + 8 * piece;
        const uint16_t* const v = p.v + (long long)b * p.Sk * p.v_stride + hk * D + 8 * piece;
        const long long begin = (long long)split * (kVectors >> p.shift);
        float2 top = make_float2(0.f, 0.f);
        // (all warps stay in the loop)
        for (long long r0 = begin; r0 < rows; r0 += 4 * step) {
            const long long r = r0 + (vector >> p.shift);
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long at = r + i * step;
                const uint16_t* from = v + (at - q_rows) * p.v_stride;
                if (at < q_rows) {
                    const long long token = at <= 0x7fffffff ? (long long)((unsigned)at / (unsigned)p.group) : at / p.group;
                    from = d_o + (token * p.Hkv * p.group + (at - token * p.group)) * D;
                }
                w[i] = at < rows ? __ldcg(reinterpret_cast<const uint4*>(from)) : make_uint4(0u, 0u, 0u, 0u);
            }
            // four sums over a vector's lanes, each in the end in a quarter of them: 4 or 5 exchanges instead of 12 or 16
            float s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = squares(w[2 * i]), c = squares(w[2 * i + 1]);
                s[i] = (lane & 1 ? c : a) + __shfl_xor_sync(0xffffffffu, lane & 1 ? a : c, 1);
            }
            float t = (lane & 2 ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, lane & 2 ? s[0] : s[1], 2);
#pragma unroll
            for (int d = 4; d < kLanes; d *= 2) t += __shfl_xor_sync(0xffffffffu, t, d);
            if (r + (lane & 3) * step < q_rows) top.x = fmaxf(top.x, t);
            else top.y = fmaxf(top.y, t);
        }
        auto over = [&](int lanes) {
            for (int d = lanes / 2; d > 0; d >>= 1) {
                top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, d));
                top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, d));
            }
        };
        over(4);
        if (piece == 0) part[vector] = top;
        __syncthreads();
        const int head = threadIdx.x / 32;                        // a warp each
        if (head < heads) {
            top = make_float2(0.f, 0.f);
            for (int e = head + lane * heads; e < kVectors; e += 32 * heads) {
                const float2 x = part[e];
                top = make_float2(fmaxf(top.x, x.x), fmaxf(top.y, x.y));
            }
            over(32);
            if (lane == 0)
                p.range[((long long)at_heads * heads + head) * p.parts + split] =
                    __float_as_uint(top.x) >> 16 | (__float_as_uint(top.y) & 0xffff0000u);
        }
        __syncthreads();
    }
}

// Eight values a thread: bound by the parts' reads, which come from L2.
template <bool BF16>
__global__ void __launch_bounds__(256) bwd_join_kernel(const JoinParams a, const JoinParams b) {
    wait_for_inputs();
    let_next_start();
    const JoinParams& p = blockIdx.y == 0 ? a : b;
    const long long n = p.tokens * (p.width / 8);
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < n; e += (long long)gridDim.x * 256) {
        float x[8] = {};
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            const float4* src = reinterpret_cast<const float4*>(p.part + s * p.apart + 8 * e);
            const float4 u = __ldcg(src), v = __ldcg(src + 1);
            x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
            x[4] += v.x, x[5] += v.y, x[6] += v.z, x[7] += v.w;
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = x[2 * i] * p.factor, hi = x[2 * i + 1] * p.factor;
            w[i] = BF16 ? ptx::pack_bf16x2(lo, hi) : ptx::pack_f16x2(lo, hi);
        }
        const long long token = e / (p.width / 8);
        const long long row = token + token / p.rows * (p.out_rows - p.rows);
        *reinterpret_cast<uint4*>(p.out + row * p.stride + 8 * (e - token * (p.width / 8))) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

int launch_join(const JoinParams* p, int n, bool bf16, int num_sms, cudaStream_t stream) {
    const long long work = p[0].tokens * (p[0].width / 8);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::max(1LL, std::min((work + 255) / 256, 8LL * num_sms)), (unsigned)n);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bf16 ? bwd_join_kernel<true> : bwd_join_kernel<false>, p[0], p[n - 1]) == cudaSuccess
               ? ATTN_OK : ATTN_ERR_CUDA;
}

int launch_begin(unsigned int* counters, cudaStream_t stream) {
    return launch_early(bwd_begin_kernel, 1u, 32u, (size_t)0, stream, counters) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int launch_range(const RangeParams& p, int D, int num_sms, cudaStream_t stream) {
    const unsigned grid = (unsigned)std::min(p.units, 2 * num_sms);
    return launch_early(D == 128 ? bwd_range_kernel<128> : bwd_range_kernel<64>, grid, (unsigned)kRangeThreads, (size_t)0,
                        stream, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace bwd
}  // namespace attn
