// The backward kernels for fp16 at head dimension 128.
#include "bwd_inst.cuh"

ATTN_INSTANTIATE_BWD(128, false)
