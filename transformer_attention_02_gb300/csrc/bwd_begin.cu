// The kernel before the products of the attention's backward pass: it sets the
// two counters from which their CTAs take work tiles.
#include "../../include/attn.h"
#include "bwd_params.h"
#include "early_launch.h"

namespace attn {
namespace bwd {
namespace {

__global__ void bwd_begin_kernel(unsigned int* counters) {
    wait_for_inputs();
    let_next_start();
    if (threadIdx.x < 2) counters[threadIdx.x] = 0u;
}

}  // namespace

int launch_begin(unsigned int* counters, cudaStream_t stream) {
    return launch_early(bwd_begin_kernel, 1u, 32u, (size_t)0, stream, counters) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace bwd
}  // namespace attn
