// Attention over an e4m3 paged cache.
#include "paged_attn.cuh"

template int attn::paged::launch_attend<attn::paged::kE4m3>(bool (&)[2][4], const attn::paged::AttendParams&, int,
                                                       cudaStream_t);
