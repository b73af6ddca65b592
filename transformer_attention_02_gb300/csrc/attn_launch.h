// Host-side launchers of the compiled forward-kernel variants.
//
// Each variant (head dimension, causal mask, additive mask, 16-bit type,
// rotary embedding of the queries, GQA head packing, window, ragged lengths) is compiled in one of the fwd_*.cu
// translation units, so that the variants build in parallel; the C ABI in
// attn_api.cu reaches them only through launch_fwd.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

struct FwdParams;

// Launches attn_fwd_kernel<D, CAUSAL, ADDITIVE, BF16, ROPE, PACK, WINDOW, RAGGED> with `grid`
// CTAs on `stream` (tensor maps of Q, K, V and of the output O, which the
// kernel stores through for the upper sub-tiles when it writes 16-bit O). `attr_set` caches, per device, that the
// variant's shared-memory attribute has been set and its register count
// checked (the in-kernel register split needs exactly the launch count).
// Returns ATTN_OK, ATTN_ERR_UNSUPPORTED (register count differs) or
// ATTN_ERR_CUDA.
template <int D, bool CAUSAL, bool ADDITIVE, bool BF16, bool ROPE, bool PACK, bool WINDOW = false,
          bool RAGGED = false>
int launch_fwd(bool& attr_set, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
               const CUtensorMap& to, const FwdParams& p, int grid, cudaStream_t stream);

// Process-unique id of the current CUDA context (the current device's primary
// context is made current first when no context is). Per-context caches of the
// library are keyed by it. Returns ATTN_OK or ATTN_ERR_CUDA.
int current_context_id(unsigned long long* id);

// What the entry points outside attn_api.cu need of the current context.
struct DeviceState {
    int num_sms;
    unsigned int* status;                 // run-time status word
    bool (*paged_attr_set)[2][4];         // [cache type]: see paged::launch_attend
};

// Fills `out` for the current context. Returns ATTN_OK, ATTN_ERR_UNSUPPORTED
// (not an sm_103 device) or ATTN_ERR_CUDA.
int device_state(DeviceState* out);

// Causal attention with a window (at most 2^30; sinks >= 0) over contiguous
// tensors of capacity Sk whose lengths differ by sequence and are read on the
// device: kv_lens (B), and q_lens (B) or null. Rows at or past a sequence's
// queries are not written; V must be finite up to the next multiple of 128 keys.
// The keys come from pages of 2^page_shift: those whose entry in block_table (B, Sk >>
// page_shift) is not one of n_pages are hidden.
// Other arguments as for attn_fwd.
int launch_ragged(const void* q, long long q_stride, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                  int Hkv, int Sq, int Sk, int D, float scale, int window, int sinks, const int* kv_lens,
                  const int* q_lens, const int* block_table, int page_shift, int n_pages, cudaStream_t stream, bool bf16);

// SM count of the current device (148 when it cannot be read, e.g. no GPU).
int device_sm_count();

}  // namespace attn
