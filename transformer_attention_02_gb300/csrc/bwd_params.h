// Host-visible parameters of the attention's backward kernels and their
// launchers (bwd_small.cu, bwd_inst.cuh).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace attn {
namespace bwd {

constexpr int kBlock = 128;         // queries and keys of a tile
constexpr int kMostRanges = 160;    // blocks of launch_range

// Rows of the row statistics: whole blocks of queries for each (b, query head).
inline long long padded_rows(int Sq) { return ((long long)Sq + kBlock - 1) / kBlock * kBlock; }

struct BwdParams {
    const uint16_t* o;              // (B, Sq, Hq, D) contiguous
    const float* lse;               // (B, Hq, Sq)
    // (B, Hq, Sp) FP32, Sp = padded_rows(Sq), from the dQ kernel to the other one; a row that is none holds -inf and 0
    float* neg_lse;                 // -lse in log2 units; with an additive mask: -(row maximum)
    float* neg_delta;               // -sum_d dO O (in fp16 times what dS carries more than P)
    float* inv_sum;                 // additive mask only: 1 / row sum
    const float* mask;              // (B, Sq, Sk) FP32 or null
    void *dq, *dk, *dv;             // gradients in the inputs' type
    long long dq_stride, dk_stride, dv_stride;   // elements from token to token
    int B, Hq, Hkv, Sq, Sk, Sp;
    int group;                      // Hq / Hkv
    int n_qb, n_kb;                 // blocks of 128 queries, of 128 keys
    int sink_kb;                    // the first key blocks, which hold a window's sinks
    int off;                        // Sk - Sq: query i sits at position i + off
    int causal, window, sinks;      // window 0: none (causal with it)
    int splits;                     // parts of a tile's walk, each a tile of its own (not dQ with an additive mask)
    int cut;                        // dK and dV, splits > 1: the first `cut` tiles are in parts, those of the first part_rows keys
    int part_rows;
    float* part;                    // splits > 1: FP32 sums of the parts, [splits] (B, Sq, Hq, D) or [splits][dV, dK] (B, part_rows, Hkv, D)
    int n_tiles;                    // tiles, each part one
    unsigned int* counter;          // tiles handed out beyond each CTA's first; launch_begin or launch_range sets it to 0
    const unsigned int* range;      // fp16: of each block of launch_range, max |dO| and, in the upper half, max |V|
    int n_range;
    int vec8;                       // gradients may be written with 32-byte stores
    int stall;                      // failure-detection test hook, as in the forward kernel
    float scale, scale_log2;
    unsigned long long timeout_ns;
    unsigned int* status;
};

// The sum of a tensor's parts, times a factor, to 16 bits.
struct JoinParams {
    const float* part;              // the tensor's first part
    long long apart;                // values from part to part
    int splits;
    uint16_t* out;                  // (B, out_rows, width), `stride` from token to token; the first `rows` of each batch item
    long long tokens, stride;       // B * rows
    int rows, out_rows;
    int width;
    float factor;
};

// Launchers; ATTN_OK or ATTN_ERR_CUDA. attr_set: per context and variant, that the shared memory is set of the kernel of
// whole walks, of the one of parts.
int launch_begin(unsigned int* counters, cudaStream_t stream);        // two of them to 0
// fp16: the same, and the largest finite |dO| ((tokens, width) contiguous) and |V| (v_stride from token to token) that each of
// `blocks` blocks finds, as two 16-bit halves.
int launch_range(unsigned int* counters, unsigned int* range, int blocks, const void* d_o, long long q_values, const void* v,
                 long long kv_tokens, long long v_stride, int kv_width, cudaStream_t stream);
int launch_join(const JoinParams* p, int n, bool bf16, int num_sms, cudaStream_t stream);        // one or two tensors
template <int D, bool BF16, bool ADDITIVE>
int launch_dq(bool* attr_set, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& d_o,
              const BwdParams& p, int grid, cudaStream_t stream);
template <int D, bool BF16, bool ADDITIVE>
int launch_dkv(bool* attr_set, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& d_o,
               const BwdParams& p, int grid, cudaStream_t stream);

}  // namespace bwd
}  // namespace attn
