// Rotary positions with several axes (time, height and width of images and
// video): the pairs of a head vector are dealt out to the axes in order, and a
// pair turns by the angle of its own axis's position. With the table's entry
// (pos, i) = {cos, sin} of pos * f_i, pair i of axis a becomes
//   (x0, x1) -> (x0 cos - x1 sin, x1 cos + x0 sin),  (pos, i) = (positions[token][a], i),
// in FP32, rounded once. With the opposite angle (inverse) it is the way back of
// a gradient: a rotation's transpose.
//
// Queries and keys go through one launch. A warp takes a token, or some of its
// heads where there are few tokens; when a head vector's 16-byte pieces (four
// pairs) divide 32, a lane always meets the same piece, so it fetches its four
// pairs' angles once for all heads. Bound by memory: every value is read and
// written once. Measured: 4 x 4097 tokens of 32 / 8 heads of 128 inside a
// packed projection 54 us, 6.2 TB/s (93% of a copy); a step of 32 single tokens 6 us, most of it the call's.
#include <algorithm>

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "attn_launch.h"
#include "paged_params.h"

namespace attn {
namespace {

constexpr int kMaxAxes = 4;
constexpr int kPieces = 4;              // 16-byte pieces of a lane in flight

struct AxesParams {
    const uint16_t* x[2];               // queries, keys
    uint16_t* y[2];
    long long x_stride[2], y_stride[2];
    int heads[2];
    const int* positions;               // (tokens, axes)
    const float2* table;                // (max_pos, D / 2)
    long long tokens;
    int max_pos, D, axes;
    int end[kMaxAxes];                  // first pair behind each axis's
    int parts, part_heads;              // units of a token, heads of a unit
    int shift;                          // log2(D / 8) where that is a power of two
    float sign;                         // -1: the opposite angle
    unsigned int* status;
};

struct Angles {
    float c[4], s[4];
};

__device__ __forceinline__ Angles angles_of(const AxesParams& p, int piece, const int (&pos)[kMaxAxes]) {
    Angles a;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int pair = 4 * piece + e;
        int at = pos[0];
#pragma unroll
        for (int k = 1; k < kMaxAxes; ++k)
            if (k < p.axes && pair >= p.end[k - 1]) at = pos[k];
        const float2 t = __ldg(p.table + (long long)at * (p.D / 2) + pair);
        a.c[e] = t.x;
        a.s[e] = t.y * p.sign;
    }
    return a;
}

template <bool BF16>
__device__ __forceinline__ uint4 turn(const uint4& w, const Angles& a) {
    return make_uint4(rotate_pair<BF16>(w.x, a.c[0], a.s[0]), rotate_pair<BF16>(w.y, a.c[1], a.s[1]),
                      rotate_pair<BF16>(w.z, a.c[2], a.s[2]), rotate_pair<BF16>(w.w, a.c[3], a.s[3]));
}

// FIXED: the pieces of a head vector divide 32.
template <bool BF16, bool FIXED>
__global__ void __launch_bounds__(256) rope_axes_kernel(const AxesParams p) {
    wait_for_inputs();
    let_next_start();
    const int lane = threadIdx.x & 31;
    const int pieces = p.D / 8;                               // of a head vector
    const long long units = p.tokens * p.parts;
    const long long warps = (long long)gridDim.x * 8;
    for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += warps) {
        const long long token = u / p.parts;
        const int h0 = (int)(u - token * p.parts) * p.part_heads, h1 = min(h0 + p.part_heads, p.heads[0] + p.heads[1]);
        int pos[kMaxAxes];
        bool ok = true;
#pragma unroll
        for (int k = 0; k < kMaxAxes; ++k) {
            pos[k] = 0;
            if (k < p.axes) {
                pos[k] = p.positions[token * p.axes + k];
                ok &= (unsigned)pos[k] < (unsigned)p.max_pos;
            }
        }
        if (!ok) {                                            // the token is left as it is
            if (lane == 0) atomicOr(p.status, paged::kStatusBadIndex);
            continue;
        }
        Angles a;
        if (FIXED) a = angles_of(p, lane & (pieces - 1), pos);
        const int n = (h1 - h0) * pieces;
        auto where = [&](int j, int& piece, int& which) -> long long {          // elements into the token's row
            const int h = h0 + (FIXED ? j >> p.shift : j / pieces);
            piece = FIXED ? j & (pieces - 1) : j % pieces;
            which = h >= p.heads[0];
            return (long long)(which ? h - p.heads[0] : h) * p.D + 8 * piece;
        };
        for (int j0 = lane; j0 < n; j0 += 32 * kPieces) {
            uint4 w[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int j = j0 + 32 * i;
                int piece, which;
                if (j < n) {
                    const long long at = where(j, piece, which);
                    w[i] = __ldcg(reinterpret_cast<const uint4*>(p.x[which] + token * p.x_stride[which] + at));
                }
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int j = j0 + 32 * i;
                int piece, which;
                if (j < n) {
                    const long long at = where(j, piece, which);
                    if (!FIXED) a = angles_of(p, piece, pos);
                    *reinterpret_cast<uint4*>(p.y[which] + token * p.y_stride[which] + at) = turn<BF16>(w[i], a);
                }
            }
        }
    }
}

// Table of the angles with frequencies of each axis's own: pair j of an axis of n pairs turns by pos * base^(-j / n).
__global__ void axes_table_kernel(float2* table, int max_pos, int pairs, int axes, int4 end, double base) {
    const int e[kMaxAxes] = {end.x, end.y, end.z, end.w};
    const long long n = (long long)max_pos * pairs;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long pos = i / pairs;
        const int pair = (int)(i - pos * pairs);
        int from = 0, to = e[0];
        for (int k = 1; k < axes; ++k)
            if (pair >= e[k - 1]) from = e[k - 1], to = e[k];
        double sn, cs;
        sincos((double)pos * pow(base, -(double)(pair - from) / (to - from)), &sn, &cs);
        table[i] = make_float2((float)cs, (float)sn);
    }
}

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// The axes' ends; false unless 1 to 4 axes hold `pairs` pairs together.
bool axes_ok(const int* sections, int axes, int pairs, int* end) {
    if (!sections || axes < 1 || axes > kMaxAxes) return false;
    long long at = 0;
    for (int k = 0; k < axes; ++k) {
        if (sections[k] < 0) return false;
        at += sections[k];
        if (at > pairs) return false;
        end[k] = (int)at;
    }
    return at == pairs;
}

bool rows_ok(const void* x, const void* y, long long xs, long long ys, long long tokens, int H, int D) {
    if (tokens == 0 || H == 0) return true;
    return x && y && aligned(x, 16) && aligned(y, 16) && xs >= (long long)H * D && ys >= (long long)H * D && xs % 8 == 0 && ys % 8 == 0;
}

int rope_axes_impl(const void* q, void* q_out, long long q_stride, long long q_out_stride, const void* k, void* k_out,
                   long long k_stride, long long k_out_stride, int B, int S, int Hq, int Hkv, int D, const float* table,
                   int max_pos, const int* positions, const int* sections, int n_axes, int inverse, cudaStream_t stream,
                   bool bf16) {
    if (B < 0 || S < 0 || Hq < 0 || Hkv < 0 || D <= 0 || D % 8 != 0 || D > 1024 || max_pos <= 0) return ATTN_ERR_INVALID_ARG;
    if ((long long)Hq + Hkv > 0x7fffffffLL / D) return ATTN_ERR_INVALID_ARG;
    AxesParams p{};
    if (!axes_ok(sections, n_axes, D / 2, p.end)) return ATTN_ERR_INVALID_ARG;
    const long long tokens = (long long)B * S;
    if (!rows_ok(q, q_out, q_stride, q_out_stride, tokens, Hq, D) || !rows_ok(k, k_out, k_stride, k_out_stride, tokens, Hkv, D))
        return ATTN_ERR_INVALID_ARG;
    if (tokens == 0 || Hq + Hkv == 0) return ATTN_OK;
    // In place is each on its own place; a result where the other tensor is read, or written, is none.
    if (Hq > 0 && tokens > 1 && q == q_out && q_stride != q_out_stride) return ATTN_ERR_INVALID_ARG;
    if (Hkv > 0 && tokens > 1 && k == k_out && k_stride != k_out_stride) return ATTN_ERR_INVALID_ARG;
    if (Hq > 0 && Hkv > 0 && (q_out == k_out || q_out == k || k_out == q)) return ATTN_ERR_INVALID_ARG;
    if (!table || !aligned(table, 8) || !positions || !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
    DeviceState dev{};
    const int rc = device_state(&dev);
    if (rc != ATTN_OK) return rc;
    p.x[0] = static_cast<const uint16_t*>(q);
    p.x[1] = static_cast<const uint16_t*>(k);
    p.y[0] = static_cast<uint16_t*>(q_out);
    p.y[1] = static_cast<uint16_t*>(k_out);
    p.x_stride[0] = q_stride, p.x_stride[1] = k_stride;
    p.y_stride[0] = q_out_stride, p.y_stride[1] = k_out_stride;
    p.heads[0] = Hq, p.heads[1] = Hkv;
    p.positions = positions;
    p.table = reinterpret_cast<const float2*>(table);
    p.tokens = tokens;
    p.max_pos = max_pos;
    p.D = D;
    p.axes = n_axes;
    p.sign = inverse ? -1.f : 1.f;
    p.status = dev.status;
    // A warp takes a whole token's heads where that gives every SM its 32 warps; with fewer tokens, down to the heads of
    // one round of loads.
    const int heads = Hq + Hkv, least = std::max(1, 32 * kPieces / (D / 8));
    const long long want = std::max(1LL, (32LL * dev.num_sms + tokens - 1) / tokens);
    p.part_heads = (int)std::max<long long>(least, (heads + want - 1) / want);
    p.parts = (heads + p.part_heads - 1) / p.part_heads;
    const long long units = tokens * p.parts;
    const unsigned grid = (unsigned)std::max(1LL, std::min((units + 7) / 8, 8LL * dev.num_sms));
    auto run = [&](auto kernel) {
        return launch_early(kernel, grid, 256u, (size_t)0, stream, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    };
    const bool fixed = 32 % (D / 8) == 0;
    while ((8 << p.shift) < D) ++p.shift;
    if (bf16) return fixed ? run(rope_axes_kernel<true, true>) : run(rope_axes_kernel<true, false>);
    return fixed ? run(rope_axes_kernel<false, true>) : run(rope_axes_kernel<false, false>);
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_rope_axes(const void* q, void* q_out, long long q_stride, long long q_out_stride, const void* k, void* k_out,
                   long long k_stride, long long k_out_stride, int B, int S, int Hq, int Hkv, int D, const float* rope_table,
                   int max_pos, const int* positions, const int* sections, int n_axes, int inverse, attn_stream_t stream) {
    return attn::rope_axes_impl(q, q_out, q_stride, q_out_stride, k, k_out, k_stride, k_out_stride, B, S, Hq, Hkv, D, rope_table,
                                max_pos, positions, sections, n_axes, inverse, reinterpret_cast<cudaStream_t>(stream), true);
}

int attn_rope_axes_f16(const void* q, void* q_out, long long q_stride, long long q_out_stride, const void* k, void* k_out,
                       long long k_stride, long long k_out_stride, int B, int S, int Hq, int Hkv, int D,
                       const float* rope_table, int max_pos, const int* positions, const int* sections, int n_axes,
                       int inverse, attn_stream_t stream) {
    return attn::rope_axes_impl(q, q_out, q_stride, q_out_stride, k, k_out, k_stride, k_out_stride, B, S, Hq, Hkv, D, rope_table,
                                max_pos, positions, sections, n_axes, inverse, reinterpret_cast<cudaStream_t>(stream), false);
}

int attn_rope_axes_table(float* table, int max_pos, const int* sections, int n_axes, double base, attn_stream_t stream) {
    int end[attn::kMaxAxes] = {};
    long long pairs = 0;
    if (!sections || n_axes < 1 || n_axes > attn::kMaxAxes || max_pos < 0 || !(base > 1.0)) return ATTN_ERR_INVALID_ARG;
    for (int k = 0; k < n_axes; ++k) {
        if (sections[k] < 0) return ATTN_ERR_INVALID_ARG;
        pairs += sections[k];
    }
    if (pairs < 1 || pairs > 512 || !attn::axes_ok(sections, n_axes, (int)pairs, end) || max_pos * pairs > 1LL << 30)
        return ATTN_ERR_INVALID_ARG;
    if (max_pos == 0) return ATTN_OK;
    if (!table || !attn::aligned(table, 16)) return ATTN_ERR_INVALID_ARG;
    attn::DeviceState dev{};
    const int rc = attn::device_state(&dev);
    if (rc != ATTN_OK) return rc;
    const long long n = max_pos * pairs;
    const unsigned grid = (unsigned)std::max(1LL, std::min((n + 255) / 256, 8LL * dev.num_sms));
    attn::axes_table_kernel<<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<float2*>(table), max_pos, (int)pairs, n_axes, make_int4(end[0], end[1], end[2], end[3]), base);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
