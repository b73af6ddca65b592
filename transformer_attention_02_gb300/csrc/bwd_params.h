// Host-visible parameters of the attention's backward kernels and their
// launchers (bwd_small.cu, bwd_inst.cuh).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace attn {
namespace bwd {

constexpr int kBlock = 128;         // queries and keys of a tile
constexpr int kRangeThreads = 512;  // of a block of launch_range

// Rows of the row statistics: whole blocks of queries for each (b, query head).
inline long long padded_rows(int Sq) { return ((long long)Sq + kBlock - 1) / kBlock * kBlock; }

struct BwdParams {
    const uint16_t* o;              // (B, Sq, Hq, D) contiguous
    const float* lse;               // (B, Hq, Sq)
    // (B, Hq, Sp) FP32, Sp = padded_rows(Sq), from the dQ kernel to the other one
    float* neg_lse;                 // -lse in log2 units (fp16: and 14, which P carries); a row that is none, or sees no key: -inf.
                                    // With an additive mask -lse, or -(row maximum) where the rows are found anew; such a row: 0
    float* neg_delta;               // -sum_d dO O (in fp16 times what dS carries more than P); a row that is none: 0
    float* inv_sum;                 // additive mask only: 1, or 1 / row sum (fp16: times 2^14); a row that is none, or sees no key: 0
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
    const unsigned int* range;      // fp16: what launch_range has left, n_range words for each (b, K/V head)
    int n_range;
    int vec8;                       // gradients may be written with 32-byte stores
    int stall;                      // failure-detection test hook, as in the forward kernel
    float scale, scale_log2;
    unsigned long long timeout_ns;
    unsigned int* status;
};

// fp16: the counters to 0, and the largest norms of dO's and V's head vectors (infinities and NaN left out) of each (b, K/V
// head), as `parts` words, which hold the upper 16 bits of the FP32 squares that a part of the tokens has: dO's low, V's high.
struct RangeParams {
    unsigned int *counters, *range;
    const uint16_t *d_o, *v;        // (B, Sq, Hkv * group, D) contiguous; (B, Sk, Hkv, D), v_stride from token to token
    long long v_stride;
    int shift;                      // a block takes 2^shift heads (a divisor of Hkv, at most 8)
    int units;                      // (B * Hkv >> shift) * parts
    int parts, Hkv, group, Sq, Sk;
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
int launch_range(const RangeParams& p, int D, int num_sms, cudaStream_t stream);
int launch_join(const JoinParams* p, int n, bool bf16, int num_sms, cudaStream_t stream);        // one or two tensors
template <int D, bool BF16, bool ADDITIVE>
int launch_dq(bool* attr_set, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& d_o,
              const BwdParams& p, int grid, cudaStream_t stream);
template <int D, bool BF16, bool ADDITIVE>
int launch_dkv(bool* attr_set, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& d_o,
               const BwdParams& p, int grid, cudaStream_t stream);

}  // namespace bwd
}  // namespace attn
