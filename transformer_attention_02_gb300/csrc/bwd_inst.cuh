// Definition of the backward kernels' launchers and the macro that instantiates
// them for one 16-bit type and head dimension in a translation unit of its own.
#pragma once

#include "bwd_kernel.cuh"

namespace attn {
namespace bwd {

template <typename Kernel>
int launch(bool& attr_set, Kernel kernel, int smem, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
           const CUtensorMap& d_o, const BwdParams& p, int grid, cudaStream_t stream) {
    if (!attr_set) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return ATTN_ERR_CUDA;
        attr_set = true;
    }
    return launch_early(kernel, (unsigned)grid, (unsigned)kThreads, (size_t)smem, stream, q, k, v, d_o, p) == cudaSuccess
               ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, bool BF16, bool ADDITIVE>
int launch_dq(bool* attr_set, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& d_o,
              const BwdParams& p, int grid, cudaStream_t stream) {
    constexpr int smem = QCfg<D, ADDITIVE>::kSmemBytes;
    if constexpr (!ADDITIVE)                              // (the statistics of a masked row need its whole walk)
        if (p.splits > 1)
            return launch(attr_set[1], bwd_dq_kernel<D, BF16, ADDITIVE, true>, smem, q, k, v, d_o, p, grid, stream);
    return launch(attr_set[0], bwd_dq_kernel<D, BF16, ADDITIVE, false>, smem, q, k, v, d_o, p, grid, stream);
}

template <int D, bool BF16, bool ADDITIVE>
int launch_dkv(bool* attr_set, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& d_o,
               const BwdParams& p, int grid, cudaStream_t stream) {
    constexpr int smem = KvCfg<D, ADDITIVE>::kSmemBytes;
    if (p.splits > 1) return launch(attr_set[1], bwd_dkv_kernel<D, BF16, ADDITIVE, true>, smem, q, k, v, d_o, p, grid, stream);
    return launch(attr_set[0], bwd_dkv_kernel<D, BF16, ADDITIVE, false>, smem, q, k, v, d_o, p, grid, stream);
}

}  // namespace bwd
}  // namespace attn

#define ATTN_BWD_ONE(LAUNCH, D, BF16, ADDITIVE)                                                               \
    template int attn::bwd::LAUNCH<D, BF16, ADDITIVE>(bool*, const CUtensorMap&, const CUtensorMap&,          \
                                                      const CUtensorMap&, const CUtensorMap&,                 \
                                                      const attn::bwd::BwdParams&, int, cudaStream_t);

#define ATTN_INSTANTIATE_BWD(D, BF16)       \
    ATTN_BWD_ONE(launch_dq, D, BF16, false)  \
    ATTN_BWD_ONE(launch_dkv, D, BF16, false) \
    ATTN_BWD_ONE(launch_dq, D, BF16, true)   \
    ATTN_BWD_ONE(launch_dkv, D, BF16, true)
