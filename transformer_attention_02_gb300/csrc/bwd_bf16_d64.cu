// The backward kernels for bf16 at head dimension 64.
#include "bwd_inst.cuh"

ATTN_INSTANTIATE_BWD(64, true)
