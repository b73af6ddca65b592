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
        const uint32_t a = x[i] & 0x7fff7fffu;
        const float2 f = widen<false>(a & ~__vcmpgeu2(a, 0x7c007c00u));
        s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
    }
    return s;
}

// A block takes a part of the tokens of one (b, K/V head), D / 8 lanes a head vector. Bound by memory, at small sizes by one
// wave's latency: two vectors of each tensor in flight.
constexpr int kRangeThreads = 512;
template <int D>
__global__ void __launch_bounds__(kRangeThreads, 2) bwd_range_kernel(const RangeParams p) {
    wait_for_inputs();
    let_next_start();
    constexpr int kLanes = D / 8, kRows = kRangeThreads / kLanes, kWarps = kRangeThreads / 32;
    __shared__ __align__(8) float part[kWarps][2];
    if (blockIdx.x == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0u;
    const int lane = threadIdx.x % 32, piece = threadIdx.x % kLanes;
    const long long q_rows = (long long)p.Sq * p.group, step = (long long)p.parts * kRows;
    for (unsigned u = blockIdx.x; u < (unsigned)p.units; u += gridDim.x) {
        const int bh = (int)(u / (unsigned)p.parts), b = bh / p.Hkv, hk = bh - b * p.Hkv;
        const uint16_t* const d_o = p.d_o + ((long long)b * p.Sq * p.Hkv + hk) * p.group * D + 8 * piece;
        const uint16_t* const v = p.v + (long long)b * p.Sk * p.v_stride + hk * D + 8 * piece;
        const long long first = ((int)u - bh * p.parts) * kRows + threadIdx.x / kLanes;
        float top = 0.f;                                          // of dO in even lanes, of V in odd ones
        // (whole warps stay in the loop: its bound is a warp's first row)
        for (long long r = first; r - lane / kLanes < max(q_rows, (long long)p.Sk); r += 2 * step) {
            uint4 w[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const long long at = r + i * step;
                w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
                if (at < q_rows) {
                    const long long token = at <= 0x7fffffff ? (long long)((unsigned)at / (unsigned)p.group) : at / p.group;
                    w[i][0] = __ldcg(reinterpret_cast<const uint4*>(
                        d_o + (token * p.Hkv * p.group + (at - token * p.group)) * D));
                }
                if (at < p.Sk) w[i][1] = __ldcg(reinterpret_cast<const uint4*>(v + at * p.v_stride));
            }
            // four sums over a vector's lanes, each in the end in a quarter of them: 4 or 5 exchanges instead of 12 or 16
            float s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = squares(w[i][0]), c = squares(w[i][1]);
                s[i] = (lane & 1 ? c : a) + __shfl_xor_sync(0xffffffffu, lane & 1 ? a : c, 1);
            }
            float t = (lane & 2 ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, lane & 2 ? s[0] : s[1], 2);
#pragma unroll
            for (int d = 4; d < kLanes; d *= 2) t += __shfl_xor_sync(0xffffffffu, t, d);
            top = fmaxf(top, t);
        }
#pragma unroll
        for (int d = 16; d > 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (lane < 2) part[threadIdx.x / 32][lane] = top;
        __syncthreads();
        if (threadIdx.x < 32) {
            const float2 both = *reinterpret_cast<const float2*>(part[lane % kWarps]);
            float o = both.x, x = both.y;
#pragma unroll
            for (int d = kWarps / 2; d > 0; d >>= 1) {
                o = fmaxf(o, __shfl_xor_sync(0xffffffffu, o, d));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            }
            if (lane == 0) p.range[u] = __float_as_uint(o) >> 16 | (__float_as_uint(x) & 0xffff0000u);
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
    const unsigned grid = (unsigned)std::min(p.units, 4 * num_sms);
    return launch_early(D == 128 ? bwd_range_kernel<128> : bwd_range_kernel<64>, grid, (unsigned)kRangeThreads, (size_t)0,
                        stream, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace bwd
}  // namespace attn
