// Forward-kernel variants in bf16 with a sliding window and sinks.
#include "attn_fwd_inst.cuh"

ATTN_INSTANTIATE_WINDOW(/*BF16=*/true, /*RAGGED=*/false)
ATTN_INSTANTIATE_WINDOW(/*BF16=*/true, /*RAGGED=*/true)
