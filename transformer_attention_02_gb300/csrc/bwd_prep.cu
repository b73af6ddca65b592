// Row statistics of the attention's backward pass: for every query row
//   delta = sum_d dO[d] O[d]      (= sum_j P_j dP_j, since O = P V),
// and the row's log-sum-exp in log2 units, both negated, as (B, Hq, Sp) with
// the rows of a head next to each other and padded to whole blocks, so that the
// products' kernels fetch 128 of them with one bulk copy. Rows that are none,
// and rows without a visible key (lse = -inf), get -inf: their probabilities
// become 2^-inf = 0.
// Bound by memory: O and dO are read once. Eight 16-byte pieces of a row a lane
// group, rows in the order in which they lie in memory.
#include <algorithm>

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "bwd_params.h"
#include "e4m3.cuh"

namespace attn {
namespace bwd {
namespace {

template <bool BF16>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = widen<BF16>(x[i]), v = widen<BF16>(y[i]);
        s0 = fmaf(u.x, v.x, s0);
        s1 = fmaf(u.y, v.y, s1);
    }
    return s0 + s1;
}

constexpr int kRows = 4;            // rows of a lane group in flight
constexpr int kSteps = 4;           // times a lane group takes kRows rows of its block's stretch

// A block takes stretches of consecutive rows, so that a row's place (b, i, h) is the stretch's first one, found by 64-bit
// divisions once, and small steps from it. Measured: 4 x 2048 tokens of 32 heads of 128 33 us, 8 x 4096 tokens 98
// us (5.5 TB/s); with 64-bit divisions for every row 45 and 160.
template <int D, bool BF16>
__global__ void __launch_bounds__(256, 4) bwd_prep_kernel(const PrepParams p) {
    constexpr int kLanes = D / 8;                        // lanes of a row
    constexpr int kGroups = 256 / kLanes;
    constexpr int kStretch = kGroups * kRows * kSteps;
    wait_for_inputs();
    let_next_start();
    if (blockIdx.x == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0u;
    const long long rows = (long long)p.B * p.Sq * p.Hq;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const uint4* o = reinterpret_cast<const uint4*>(p.o) + lane;
    const uint4* g = reinterpret_cast<const uint4*>(p.d_o) + lane;
    for (long long r0 = (long long)blockIdx.x * kStretch; r0 < rows; r0 += (long long)gridDim.x * kStretch) {
        const long long t0 = r0 / p.Hq;
        const unsigned h0 = (unsigned)(r0 - t0 * p.Hq);
        const int b0 = (int)(t0 / p.Sq);
        const unsigned i0 = (unsigned)(t0 - (long long)b0 * p.Sq);
#pragma unroll 1
        for (int step = 0; step < kSteps; ++step) {
            uint4 a[kRows], c[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const long long r = r0 + (step * kRows + u) * kGroups + group;
                a[u] = c[u] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) {
                    a[u] = __ldcg(o + r * kLanes);
                    c[u] = __ldcg(g + r * kLanes);
                }
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const unsigned at = (unsigned)((step * kRows + u) * kGroups + group);
                float s = dot8<BF16>(a[u], c[u]);
#pragma unroll
                for (int m = kLanes / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                if (lane == 0 && r0 + at < rows) {
                    const unsigned t = (h0 + at) / (unsigned)p.Hq, h = h0 + at - t * p.Hq;       // tokens on, head
                    const unsigned db = (i0 + t) / (unsigned)p.Sq, i = i0 + t - db * p.Sq;
                    const long long bh = (long long)(b0 + db) * p.Hq + h;
                    p.neg_delta[bh * p.Sp + i] = -s;
                    if (p.lse) {
                        const float l = p.lse[bh * p.Sq + i];
                        p.neg_lse[bh * p.Sp + i] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
                    }
                }
            }
        }
    }
    // rows that are none
    const int pad = p.Sp - p.Sq;
    const long long n = (long long)p.B * p.Hq * pad;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < n; e += (long long)gridDim.x * 256) {
        const long long at = e / pad * p.Sp + p.Sq + e % pad;
        p.neg_delta[at] = 0.f;
        if (p.lse) p.neg_lse[at] = -INFINITY;
    }
}

}  // namespace

int launch_prep(const PrepParams& p, bool bf16, int num_sms, cudaStream_t stream) {
    const long long per_block = 256 / (p.D / 8) * kRows * kSteps;
    const long long rows = (long long)p.B * p.Sq * p.Hq;
    const unsigned grid = (unsigned)std::max(1LL, std::min((rows + per_block - 1) / per_block, 4LL * num_sms));
    auto run = [&](auto kernel) {
        return launch_early(kernel, grid, 256u, (size_t)0, stream, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    };
    if (p.D == 128) return bf16 ? run(bwd_prep_kernel<128, true>) : run(bwd_prep_kernel<128, false>);
    return bf16 ? run(bwd_prep_kernel<64, true>) : run(bwd_prep_kernel<64, false>);
}

}  // namespace bwd
}  // namespace attn
