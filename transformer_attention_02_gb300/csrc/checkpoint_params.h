// Host-visible parameters of the 8-bit activation checkpoints (checkpoint.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace attn {
namespace checkpoint {

// A (tokens, H, D) tensor in 16 bits, `stride` elements from token to token, and its codes (contiguous) and scales.
struct Tensor {
    uint16_t* x = nullptr;
    uint8_t* codes = nullptr;
    float* scale = nullptr;
    long long stride = 0, tokens = 0;
    int H = 0;
};

// Tensors with no vector are not passed. ATTN_OK or ATTN_ERR_CUDA.
int launch_store(const Tensor& t, int D, bool bf16, int num_sms, cudaStream_t stream);
int launch_load(const Tensor* t, int n, int D, bool bf16, int num_sms, cudaStream_t stream);    // 1 to 3 tensors

}  // namespace checkpoint
}  // namespace attn
