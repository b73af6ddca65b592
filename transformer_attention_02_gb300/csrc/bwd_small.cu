// The small kernels around the products of the attention's backward pass: before
// them the two counters are set from which their CTAs take work tiles; behind
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

}  // namespace bwd
}  // namespace attn
