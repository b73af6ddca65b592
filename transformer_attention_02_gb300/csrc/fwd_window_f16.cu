// Forward-kernel variants in fp16 with a sliding window and sinks.
#include "attn_fwd_inst.cuh"

ATTN_INSTANTIATE_WINDOW(/*BF16=*/false, /*RAGGED=*/false)
ATTN_INSTANTIATE_WINDOW(/*BF16=*/false, /*RAGGED=*/true)
