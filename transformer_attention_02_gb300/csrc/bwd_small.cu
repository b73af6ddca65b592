// The small kernels around the products of the attention's backward pass: before
// them the two counters are set from which their CTAs take work tiles, and in fp16
// the largest |dO| and |V| are found, which bound dS; behind
// them, where few tiles were cut into parts, the parts' FP32 sums are joined, in
// the parts' order.
#include <algorithm>

#include "../../include/attn.h"
#include "bwd_params.h"
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

__device__ __forceinline__ uint32_t largest(uint32_t m, const uint4& w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = x[i] & 0x7fff7fffu;
        m = __vmaxu2(m, a & ~__vcmpgeu2(a, 0x7c007c00u));                    // (infinities and NaN set no range)
    }
    return m;
}

// Bound by memory, at small sizes by one wave's latency: eight values a load, two loads of each tensor in flight (13 MB: 6.8 us,
// 3.5 more than the launch it takes the place of).
constexpr int kRangeLoads = 2;
__global__ void __launch_bounds__(1024) bwd_range_kernel(unsigned int* counters, unsigned int* range, const uint4* d_o,
                                                        long long q_pieces, const uint16_t* v, long long kv_tokens,
                                                        long long v_stride, int kv_pieces) {
    wait_for_inputs();
    let_next_start();
    __shared__ uint32_t part[2][32];
    if (blockIdx.x == 0 && threadIdx.x < 2) counters[threadIdx.x] = 0u;
    const long long first = (long long)blockIdx.x * 1024 + threadIdx.x, step = (long long)gridDim.x * 1024;
    uint32_t m[2] = {0u, 0u};
    const long long pieces = kv_tokens * kv_pieces;
    const bool whole = v_stride == 8LL * kv_pieces;
    for (long long e = first; e < max(q_pieces, pieces); e += kRangeLoads * step) {
        uint4 w[kRangeLoads], x[kRangeLoads];
#pragma unroll
        for (int i = 0; i < kRangeLoads; ++i) {
            const long long at = e + i * step, token = whole || at >= pieces ? 0 : at / kv_pieces;
            w[i] = at < q_pieces ? __ldcg(d_o + at) : make_uint4(0u, 0u, 0u, 0u);
            x[i] = at < pieces ? __ldcg(reinterpret_cast<const uint4*>(v + token * v_stride + 8 * (at - token * kv_pieces)))
                               : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kRangeLoads; ++i) {
            m[0] = largest(m[0], w[i]);
            m[1] = largest(m[1], x[i]);
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m[k] = __vmaxu2(m[k], __shfl_xor_sync(0xffffffffu, m[k], d));
        if (threadIdx.x % 32 == 0) part[k][threadIdx.x / 32] = m[k];
    }
    __syncthreads();
    if (threadIdx.x < 32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[k] = part[k][threadIdx.x];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m[k] = __vmaxu2(m[k], __shfl_xor_sync(0xffffffffu, m[k], d));
            m[k] = max(m[k] & 0xffffu, m[k] >> 16);
        }
        if (threadIdx.x == 0) range[blockIdx.x] = m[0] | m[1] << 16;
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

int launch_range(unsigned int* counters, unsigned int* range, int blocks, const void* d_o, long long q_values, const void* v,
                 long long kv_tokens, long long v_stride, int kv_width, cudaStream_t stream) {
    return launch_early(bwd_range_kernel, (unsigned)blocks, 1024u, (size_t)0, stream, counters, range, static_cast<const uint4*>(d_o),
                        q_values / 8, static_cast<const uint16_t*>(v), kv_tokens, v_stride, kv_width / 8) == cudaSuccess
               ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace bwd
}  // namespace attn
