// The backward kernels for bf16 at head dimension 128.
#include "bwd_inst.cuh"

ATTN_INSTANTIATE_BWD(128, true)
