// Attention over a bf16 paged cache.
#include "paged_attn.cuh"

template int attn::paged::launch_attend<attn::paged::kBf16>(bool (&)[2][4], const attn::paged::AttendParams&, int,
                                                       cudaStream_t);
