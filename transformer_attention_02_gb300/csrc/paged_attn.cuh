// Attention of a few query rows over a paged key/value cache (16-bit, or e4m3
// with one scale per page and head):
//   s_ij = scale <rot(q_i), K_j>,  o_i = sum_j softmax_j(s_ij) V_j,
//   lse_i = log sum_j exp(s_ij),
// over the keys visible to the query at position p_i = kv_len - q_len + i:
// j <= p_i and (window = 0 or j > p_i - window or j < sinks).
//
// What bounds it: every visible key and value is read once, 2 * D bytes (8-bit)
// or 4 * D bytes a key and K/V head, for 4 * D * rows operations with 1 to 32
// rows, so the reads of the cache do. The products therefore run on mma.sync,
// whose operands come from registers: a warp takes 16 keys at a time, converts
// e4m3 codes to f16 (exact) between shared memory and the tensor cores, and
// needs no barrier with any other warp until a sequence ends. tcgen05 would
// want the converted operands written back to shared memory, and its 128-row
// tiles would hold 1 to 32 rows. The keys stand on the M axis,
//   S^T = K Q^T (16 keys x 8 rows),   O^T += V^T P^T (16 dims x 8 rows),
// so that eight query rows fill a product's N axis and a group of 4 to 8 query
// heads wastes little.
//
// Work split: the visible keys of every (sequence, K/V head, row block) are a
// list of units of 128 keys; the units of all of them, end to end, are cut into
// equal ranges, one per CTA, so that ragged batches and long contexts load
// every SM alike. A CTA that holds only part of a segment leaves its FP32
// result (unnormalised O, row maximum, row sum) in the workspace, and a second
// kernel, launched while the first one drains, merges the parts. All lengths
// are read on the device.
//
// Memory: each warp owns a ring of stages filled by 16-byte asynchronous copies
// (16 or 32 keys and their values a stage); rows that no query sees are filled
// with zeros, so whatever their slots hold never enters a product. 16-byte
// chunks are XOR-swizzled by the row, which makes the ldmatrix reads of eight
// rows conflict-free.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "paged_params.h"

namespace attn {
namespace paged {

template <int D, int CT, int NT>
struct Cfg {
    static constexpr int kElt = CT == kE4m3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElt;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kRows = 8 * NT;                         // query rows of a row block
    static constexpr int kWarps = kRowBytes == 256 ? 4 : 8;
    static constexpr int kKeys = kRowBytes == 64 ? 32 : 16;      // keys of a stage
    static constexpr int kTiles = kKeys / 16;
    static constexpr int kStageBytes = 2 * kKeys * kRowBytes;
    // Two CTAs a SM with three stages, or (32 rows: the accumulators take the
    // registers of both) one with six.
    static constexpr int kResident = NT <= 2 ? 2 : 1;
    static constexpr int kStages = NT <= 2 ? 3 : 6;
    static constexpr int kRingBytes = kStages * kStageBytes;     // of one warp
    static constexpr int kMergeStride = D + 4;                   // floats; breaks the bank alignment of the rows
    static constexpr bool kQShared = NT == 4;                    // Q fragments in shared memory, not registers
    static constexpr int kScaleOff = kWarps * kRingBytes;        // [warp][stage][tile]{k, v}
    static constexpr int kStatOff = kScaleOff + kWarps * kStages * kTiles * 8;    // [warp][row]{max, sum}
    static constexpr int kQOff = kStatOff + kWarps * kRows * 8;
    static constexpr int kSmemBytes = kQOff + (kQShared ? kRows * D * 2 : 0);
    static_assert(kRows * kMergeStride * 4 <= kRingBytes, "a warp's merge buffer reuses its ring");
    static_assert(kUnit % kKeys == 0, "a stage lies inside one unit");
    static_assert(kResident * (kSmemBytes + 1024) <= 232448, "shared memory budget");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
}

// Transposes an 8x8 matrix of 16-bit values held as an accumulator fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The two low / high e4m3 codes of a word as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ float2 widen16(uint32_t w, bool bf16) {
    float2 f;
    if (bf16) {
        f.x = __uint_as_float(w << 16);
        f.y = __uint_as_float(w & 0xffff0000u);
    } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(f.x), "=f"(f.y)
            : "r"(w));
    }
    return f;
}

// Byte offset of 16-byte chunk c of row r in a swizzled stage.
template <int ROWB>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    if (ROWB == 64) {                                            // two rows share a 128-byte line
        const int line = r >> 1;
        return (uint32_t)(line * 128 + (((((r & 1) << 2) + c) ^ (line & 7)) << 4));
    }
    return (uint32_t)(r * ROWB + ((c ^ (r & 7)) << 4));
}

// What a sequence's queries see, as a list of 128-key units: the units of the
// sinks, then those from the oldest key of the window to the last key.
struct KeyList {
    int kv, ql;          // keys in the cache, queries of the step (clamped to what the call can hold)
    int sink_units;      // units before the gap (0 when there is none)
    int first;           // the unit after them
    int units;           // length of the list
};

__device__ __forceinline__ KeyList key_list(const AttendParams& p, int b, bool& bad) {
    KeyList l;
    l.kv = p.kv_lens[b];
    l.ql = p.q_lens ? p.q_lens[b] : p.Sq;
    const long long room = (long long)p.max_pages << p.page_shift;
    bad = l.kv < 0 || l.kv > room || l.ql < 0 || l.ql > p.Sq;
    l.kv = (int)min((long long)max(l.kv, 0), room);
    l.ql = min(max(l.ql, 0), p.Sq);
    l.sink_units = l.first = l.units = 0;
    if (l.ql == 0 || l.kv == 0) return l;
    const int last = (l.kv + kUnit - 1) / kUnit;
    if (p.window > 0) {
        const int low = max(0, l.kv - l.ql - p.window + 1);      // oldest key in the first query's window
        const int su = (min(p.sinks, l.kv) + kUnit - 1) / kUnit;
        if (low / kUnit > su) {
            l.sink_units = su;
            l.first = low / kUnit;
        }
    }
    l.units = l.sink_units + last - l.first;
    return l;
}

// CTAs that work on `total` units: no more than there are units, so that every
// CTA between a segment's first and last one holds a part of it.
__device__ __forceinline__ int working_ctas(const AttendParams& p, int total) { return min(p.ctas, total); }
__device__ __forceinline__ int unit_start(int total, int ctas, int cta) { return (int)((long long)total * cta / ctas); }
// The CTA whose range holds unit x.
__device__ __forceinline__ int unit_owner(int total, int ctas, int x) {
    return (int)((((long long)x + 1) * ctas + total - 1) / total) - 1;
}

template <int D, int CT, int NT>
__global__ void __launch_bounds__(Cfg<D, CT, NT>::kWarps * 32, Cfg<D, CT, NT>::kResident)
    paged_attend_kernel(const AttendParams p) {
    using C = Cfg<D, CT, NT>;
    constexpr int kThreads = C::kWarps * 32;
    constexpr int kSteps = D / 16;                                // products of 16 dims
    constexpr bool kBf = CT == kBf16;                             // operand type of the products
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ int s_scan[kThreads / 32 + 1];
    __shared__ int s_begin[2];                                    // the CTA's first sequence and its first unit
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint8_t* ring = smem_raw + warp * C::kRingBytes;
    const uint32_t ring_a = ptx::smem_addr(ring);
    float* const scales = reinterpret_cast<float*>(smem_raw + C::kScaleOff) + warp * C::kStages * C::kTiles * 2;
    const uint32_t scales_a = ptx::smem_addr(scales);
    float2* const stats = reinterpret_cast<float2*>(smem_raw + C::kStatOff);
    uint2* const q_sh = reinterpret_cast<uint2*>(smem_raw + C::kQOff);

    // ---- where this CTA's range begins: a scan over the sequences' units
    const int segs = p.Hkv * p.row_blocks;                        // segments of a sequence
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        bool bad;
        mine += key_list(p, b, bad).units * segs;
        if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int before = incl - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int ctas = working_ctas(p, total);
    const bool works = (int)blockIdx.x < ctas;
    int x = works ? unit_start(total, ctas, blockIdx.x) : total;
    const int x_end = works ? unit_start(total, ctas, blockIdx.x + 1) : total;
    if (blockIdx.x == 0 || (before <= x && x < before + mine)) {
        int at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            bool bad;
            const int n = key_list(p, b, bad).units * segs;
            if (blockIdx.x == 0) p.base[b] = at;
            if (at <= x && x < at + n) {
                s_begin[0] = b;
                s_begin[1] = at;
            }
            at += n;
        }
        if (blockIdx.x == 0 && b_hi == p.B && b_lo < b_hi) p.base[p.B] = at;
    }
    __syncthreads();
    if (x >= x_end) return;
    int b = s_begin[0], b_base = s_begin[1];

    uint32_t qf[C::kQShared ? 1 : kSteps][C::kQShared ? 1 : NT][2];

    while (x < x_end) {
        bool bad_len;
        const KeyList list = key_list(p, b, bad_len);
        if (list.units == 0 || x >= b_base + list.units * segs) {        // the sequence is done (or empty)
            b_base += list.units * segs;
            ++b;
            continue;
        }
        const int seg = (x - b_base) / list.units;
        const int u0 = x - b_base - seg * list.units;
        const int u1 = min(list.units, u0 + x_end - x);
        const int hk = seg / p.row_blocks, rb = seg - hk * p.row_blocks;
        const int r0 = rb * C::kRows;
        const int n_keys = (u1 - u0) * kUnit;

        // Positions of the block's first and last valid rows, and what they see.
        const int i0 = r0 / p.group;
        const int i1 = min(min(p.rows - 1, r0 + C::kRows - 1) / p.group, list.ql - 1);
        const int pos_lo = list.kv - list.ql + i0, pos_hi = list.kv - list.ql + i1;
        const int kv_end = i0 < list.ql ? max(0, pos_hi + 1) : 0;        // keys at or past it: hidden from every row
        const int w_lo = p.window > 0 ? pos_lo - p.window + 1 : 0;       // keys before it are hidden, but for the sinks
        const int sinks = p.window > 0 ? p.sinks : 0;

        const int* table = p.block_table + (size_t)b * p.max_pages;
        uint32_t bad_tiles = 0;                                          // bit stage * kTiles + tile
        auto key_of = [&](int i) {                                       // first key of this warp's i-th stage, or -1
            const int off = (i * C::kWarps + warp) * C::kKeys;
            if (off >= n_keys) return -1;
            const int u = u0 + off / kUnit;
            return (u < list.sink_units ? u : u - list.sink_units + list.first) * kUnit + off % kUnit;
        };
        auto issue = [&](int i) {
            const int key0 = key_of(i);
            if (key0 >= 0 && key0 < kv_end) {
                const int s = i % C::kStages;
#pragma unroll
                for (int m = 0; m < C::kTiles; ++m) {
                    const int k0 = key0 + 16 * m;
                    int id = -1;
                    if (k0 < kv_end) {
                        id = __ldg(table + (k0 >> p.page_shift));
                        if ((unsigned)id >= (unsigned)p.n_pages) {
                            if (lane == 0) atomicOr(p.status, kStatusBadIndex);
                            id = -1;
                        }
                    }
                    const uint32_t bit = 1u << (s * C::kTiles + m);
                    bad_tiles = id < 0 ? bad_tiles | bit : bad_tiles & ~bit;
                    const size_t row0 = id < 0 ? 0
                                               : ((((size_t)id * p.Hkv + hk) << p.page_shift) +
                                                  (size_t)(k0 & ((1 << p.page_shift) - 1)));
                    const uint8_t* ks = static_cast<const uint8_t*>(p.k_cache) + row0 * C::kRowBytes;
                    const uint8_t* vs = static_cast<const uint8_t*>(p.v_cache) + row0 * C::kRowBytes;
                    const uint32_t dst = ring_a + s * C::kStageBytes;
#pragma unroll
                    for (int c = 0; c < 16 * C::kChunks / 32; ++c) {
                        const int r = (c * 32 + lane) / C::kChunks, ch = lane % C::kChunks;
                        const int key = k0 + r;
                        const bool take = id >= 0 && key < kv_end && (key >= w_lo || key < sinks);
                        const uint32_t to = swizzled<C::kRowBytes>(16 * m + r, ch);
                        const size_t from = take ? (size_t)r * C::kRowBytes + ch * 16 : 0;
                        cp_async16(dst + to, ks + from, take);
                        cp_async16(dst + C::kKeys * C::kRowBytes + to, vs + from, take);
                    }
                    if (CT == kE4m3 && lane < 2) {
                        const size_t at = id < 0 ? 0 : (size_t)id * p.Hkv + hk;
                        cp_async4(scales_a + ((s * C::kTiles + m) * 2 + lane) * 4, (lane ? p.v_scale : p.k_scale) + at);
                    }
                }
            }
            cp_async_commit();
        };
        const int n_it = (n_keys + C::kWarps * C::kKeys - 1) / (C::kWarps * C::kKeys);
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) issue(i);

        // ---- queries: rotated, rounded to their 16-bit type, as B fragments.
        // With an 8-bit cache they become f16 values, each row scaled by a
        // power of two to lie in [-2, 2]: exact down to 2^-24 of the row's
        // largest value, whatever the row's magnitude.
        float cf[NT][2];                                          // log2 units per raw score, rows 2t and 2t + 1
        auto load_q = [&](auto&& put) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = r0 + 8 * n + g;
                const int i = row / p.group;
                const bool there = row < p.rows && i < list.ql;
                int pos = list.kv - list.ql + i;
                if (p.rope && there && pos >= p.max_pos) {
                    if (t == 0) atomicOr(p.status, kStatusBadIndex);
                    pos = p.max_pos - 1;
                }
                pos = max(pos, 0);
                const uint16_t* src =
                    p.q + ((long long)b * p.Sq + i) * p.q_stride + (long long)(hk * p.group + (row - i * p.group)) * D;
                const bool bf = CT == kE4m3 ? p.q_bf16 : kBf;
                uint32_t w[kSteps][2];
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // dims of the fragment's register e: the keys' fragments hold the same ones
                        const int d = CT == kE4m3 ? 16 * s + 4 * t + 2 * e : 16 * s + 8 * e + 2 * t;
                        uint32_t v = there ? *reinterpret_cast<const uint32_t*>(src + d) : 0u;
                        if (p.rope && there) {
                            const float2 a =
                                __ldg(reinterpret_cast<const float2*>(p.rope) + (size_t)pos * (D / 2) + d / 2);
                            const float2 f = widen16(v, bf);
                            const float y0 = f.x * a.x - f.y * a.y, y1 = f.y * a.x + f.x * a.y;
                            v = bf ? ptx::pack_bf16x2(y0, y1) : ptx::pack_f16x2(y0, y1);
                        }
                        w[s][e] = v;
                        if (CT == kE4m3) {
                            const float2 f = widen16(v, bf);
                            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    }
                }
                float back = 1.f;
                if (CT == kE4m3) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -120), 120);
                    const float f = __uint_as_float((uint32_t)(127 - e) << 23);
                    back = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float2 a = widen16(w[s][h], bf);
                            w[s][h] = ptx::pack_f16x2(a.x * f, a.y * f);
                        }
                }
                cf[n][0] = p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t);
                cf[n][1] = p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) put(s, n, w[s][0], w[s][1]);
            }
        };
        if constexpr (C::kQShared) {
            load_q([&](int s, int n, uint32_t w0, uint32_t w1) {
                if (warp == 0) q_sh[(s * NT + n) * 32 + lane] = make_uint2(w0, w1);
            });
            __syncthreads();
        } else {
            load_q([&](int s, int n, uint32_t w0, uint32_t w1) {
                qf[s][n][0] = w0;
                qf[s][n][1] = w1;
            });
        }

        float acc[kSteps][NT][4];                                 // O^T
        float m_used[NT][2], l_sum[NT][2];                        // rows 2t, 2t + 1 of each n-tile; the sum is this lane's
        float v_ref = 0.f;                                        // largest value scale so far: acc is in units of it
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m_used[n][0] = m_used[n][1] = -INFINITY;
            l_sum[n][0] = l_sum[n][1] = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) acc[s][n][0] = acc[s][n][1] = acc[s][n][2] = acc[s][n][3] = 0.f;
        }

        for (int i = 0; i < n_it; ++i) {
            cp_async_wait<C::kStages - 2>();
            __syncwarp();
            issue(i + C::kStages - 1);
            const int key0 = key_of(i);
            if (key0 < 0 || key0 >= kv_end) continue;
            const int st = i % C::kStages;
#pragma unroll
            for (int m = 0; m < C::kTiles; ++m) {
                const int k0 = key0 + 16 * m;
                const bool bad = (bad_tiles >> (st * C::kTiles + m)) & 1u;
                if (bad || k0 >= kv_end) continue;
                const uint32_t ka = ring_a + st * C::kStageBytes, va = ka + C::kKeys * C::kRowBytes;
                // ---- S^T = K Q^T
                float s[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
                {
                    const int kr = 16 * m + (lane & 7) + ((lane >> 3) & 1) * 8, kc = lane >> 4;
#pragma unroll
                    for (int c = 0; c < C::kChunks / 2; ++c) {
                        uint32_t r[4];
                        ldmatrix4<false>(r, ka + swizzled<C::kRowBytes>(kr, 2 * c + kc));
                        if (CT == kE4m3) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t a0 = e4m3_lo(r[2 * h]), a1 = e4m3_lo(r[2 * h + 1]),
                                               a2 = e4m3_hi(r[2 * h]), a3 = e4m3_hi(r[2 * h + 1]);
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    uint2 q2;
                                    if constexpr (C::kQShared)
                                        q2 = q_sh[((2 * c + h) * NT + n) * 32 + lane];
                                    else
                                        q2 = make_uint2(qf[2 * c + h][n][0], qf[2 * c + h][n][1]);
                                    mma16816<false>(s[n], a0, a1, a2, a3, q2.x, q2.y);
                                }
                            }
                        } else {
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint2 q2;
                                if constexpr (C::kQShared)
                                    q2 = q_sh[(c * NT + n) * 32 + lane];
                                else
                                    q2 = make_uint2(qf[c][n][0], qf[c][n][1]);
                                mma16816<kBf>(s[n], r[0], r[1], r[2], r[3], q2.x, q2.y);
                            }
                        }
                    }
                }
                // ---- logits in log2 units; hidden keys to -inf
                float ks = 1.f, vs = 1.f;
                if (CT == kE4m3) {
                    const float2 kv2 = *reinterpret_cast<const float2*>(scales + (st * C::kTiles + m) * 2);
                    ks = kv2.x;
                    vs = kv2.y;
                }
                const bool whole = k0 + 15 <= pos_lo && (k0 >= pos_hi - p.window + 1 || p.window == 0 || k0 + 16 <= sinks);
                bool grow = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = cf[n][e] * ks;
                        float z0 = s[n][e] * f, z1 = s[n][2 + e] * f;
                        if (!whole) {
                            const int pos = list.kv - list.ql + (r0 + 8 * n + 2 * t + e) / p.group;
                            const int lo = p.window > 0 ? pos - p.window : -1;
                            const int j0 = k0 + g, j1 = j0 + 8;
                            if (j0 > pos || (j0 <= lo && j0 >= sinks)) z0 = -INFINITY;
                            if (j1 > pos || (j1 <= lo && j1 >= sinks)) z1 = -INFINITY;
                        }
                        s[n][e] = z0;
                        s[n][2 + e] = z1;
                        grow |= fmaxf(z0, z1) > m_used[n][e] + kRescaleThreshold;
                    }
                }
                // The maximum in use may trail the true one by 2^8 (the weights
                // then reach 2^8, far inside 16-bit range), so most tiles need
                // one vote instead of the reduction and the rescaling.
                if (__any_sync(0xffffffffu, grow) || vs > v_ref) {
                    const float fv = vs > v_ref ? v_ref / vs : 1.f;
                    v_ref = fmaxf(v_ref, vs);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                            mx = fmaxf(mx, m_used[n][e]);
                            const float alpha = mx == -INFINITY ? 1.f : ptx::ex2(m_used[n][e] - mx);
                            m_used[n][e] = mx;
                            l_sum[n][e] *= alpha;
                            const float f = alpha * fv;
#pragma unroll
                            for (int d = 0; d < kSteps; ++d) {
                                acc[d][n][e] *= f;
                                acc[d][n][2 + e] *= f;
                            }
                        }
                    }
                }
                // ---- weights; P in f16 (bf16 for a bf16 cache), summed before that rounding
                const float vf = CT == kE4m3 ? (v_ref > 0.f ? vs / v_ref : 0.f) : 1.f;
                uint32_t pb[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float nm = m_used[n][e] == -INFINITY ? 0.f : m_used[n][e];
                        w[e] = ptx::ex2(s[n][e] - nm);
                        w[2 + e] = ptx::ex2(s[n][2 + e] - nm);
                        l_sum[n][e] += w[e] + w[2 + e];
                    }
                    if (CT == kE4m3) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] *= vf;
                    }
                    pb[n][0] = transpose8x8(kBf ? ptx::pack_bf16x2(w[0], w[1]) : ptx::pack_f16x2(w[0], w[1]));
                    pb[n][1] = transpose8x8(kBf ? ptx::pack_bf16x2(w[2], w[3]) : ptx::pack_f16x2(w[2], w[3]));
                }
                // ---- O^T += V^T P^T
                {
                    const int vr = 16 * m + (lane & 7) + (lane >> 4) * 8, vc = (lane >> 3) & 1;
#pragma unroll
                    for (int c = 0; c < C::kChunks / 2; ++c) {
                        uint32_t r[4];
                        ldmatrix4<true>(r, va + swizzled<C::kRowBytes>(vr, 2 * c + vc));
                        if (CT == kE4m3) {
                            // Each register holds two keys of two neighbouring dims: the even
                            // dims of both chunks make one product, the odd ones the other.
#pragma unroll
                            for (int j = 0; j < 4; ++j) r[j] = __byte_perm(r[j], 0u, 0x3120);
                            const uint32_t e0 = e4m3_lo(r[0]), e1 = e4m3_lo(r[1]), e2 = e4m3_lo(r[2]), e3 = e4m3_lo(r[3]);
                            const uint32_t o0 = e4m3_hi(r[0]), o1 = e4m3_hi(r[1]), o2 = e4m3_hi(r[2]), o3 = e4m3_hi(r[3]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma16816<false>(acc[2 * c][n], e0, e1, e2, e3, pb[n][0], pb[n][1]);
                                mma16816<false>(acc[2 * c + 1][n], o0, o1, o2, o3, pb[n][0], pb[n][1]);
                            }
                        } else {
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma16816<kBf>(acc[c][n], r[0], r[1], r[2], r[3], pb[n][0], pb[n][1]);
                        }
                    }
                }
            }
        }

        // ---- merge the warps: each leaves its O^T (times its value scale), its
        // maximum and its sum in shared memory
        cp_async_wait<0>();
        __syncwarp();
        float* const mine_o = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = 8 * n + 2 * t + e;
                float l = l_sum[n][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (g == 0) stats[warp * C::kRows + col] = make_float2(m_used[n][e], l);
                const float f = CT == kE4m3 ? v_ref : 1.f;
#pragma unroll
                for (int d = 0; d < kSteps; ++d) {
                    const int da = CT == kE4m3 ? 32 * (d >> 1) + (d & 1) + 2 * g : 16 * d + g;
                    const int db = CT == kE4m3 ? da + 16 : da + 8;
                    mine_o[col * C::kMergeStride + da] = acc[d][n][e] * f;
                    mine_o[col * C::kMergeStride + db] = acc[d][n][2 + e] * f;
                }
            }
        }
        __syncthreads();
        const bool full = u0 == 0 && u1 == list.units;
        float* slot = p.part + (size_t)(2 * blockIdx.x + (u0 == 0 ? 1 : 0)) * C::kRows * (D + 2);
        for (int w = tid; w < C::kRows * (D / 4); w += kThreads) {
            const int col = w / (D / 4), d = (w - col * (D / 4)) * 4;
            float mx = -INFINITY;
#pragma unroll
            for (int v = 0; v < C::kWarps; ++v) mx = fmaxf(mx, stats[v * C::kRows + col].x);
            float sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mx != -INFINITY) {
#pragma unroll
                for (int v = 0; v < C::kWarps; ++v) {
                    const float2 st2 = stats[v * C::kRows + col];
                    const float f = ptx::ex2(st2.x - mx);
                    const float4 a = *reinterpret_cast<const float4*>(
                        reinterpret_cast<const float*>(smem_raw + v * C::kRingBytes) + col * C::kMergeStride + d);
                    if (st2.x != -INFINITY) {
                        sum += st2.y * f;
                        o.x = fmaf(a.x, f, o.x);
                        o.y = fmaf(a.y, f, o.y);
                        o.z = fmaf(a.z, f, o.z);
                        o.w = fmaf(a.w, f, o.w);
                    }
                }
            }
            if (full) {
                const int row = r0 + col, i = row / p.group;
                if (row < p.rows && i < list.ql) {
                    const int h = hk * p.group + (row - i * p.group);
                    const float inv = sum > 0.f ? 1.f / sum : 0.f;
                    const bool bf = CT == kE4m3 ? p.q_bf16 : kBf;
                    uint2 r;
                    r.x = bf ? ptx::pack_bf16x2(o.x * inv, o.y * inv) : ptx::pack_f16x2(o.x * inv, o.y * inv);
                    r.y = bf ? ptx::pack_bf16x2(o.z * inv, o.w * inv) : ptx::pack_f16x2(o.z * inv, o.w * inv);
                    *reinterpret_cast<uint2*>(p.o + (((size_t)b * p.Sq + i) * p.Hq + h) * D + d) = r;
                    if (d == 0)
                        p.lse[((size_t)b * p.Hq + h) * p.Sq + i] =
                            sum > 0.f ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
                }
            } else {
                *reinterpret_cast<float4*>(slot + col * D + d) = o;
                if (d == 0) {
                    slot[C::kRows * D + col] = mx;
                    slot[C::kRows * (D + 1) + col] = sum;
                }
            }
        }
        __syncthreads();                                          // the rings are free for the next segment
        x += u1 - u0;
    }
}

// Merges the parts of the segments that several CTAs share, and fills the rows
// of sequences without a key. One warp per row; a lane holds D / 32 dims.
template <int D, int RB>
__global__ void __launch_bounds__(256) paged_merge_kernel(const AttendParams p, bool bf16) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int segs = p.Hkv * p.row_blocks;
    const int b = blockIdx.x / segs, seg = blockIdx.x - b * segs;
    const int total = p.base[p.B], first = p.base[b];
    const int units = (p.base[b + 1] - first) / segs;
    int c0 = 0, c1 = 0;
    if (units > 0) {
        const int ctas = working_ctas(p, total);
        c0 = unit_owner(total, ctas, first + seg * units);
        c1 = unit_owner(total, ctas, first + (seg + 1) * units - 1);
        if (c0 == c1) return;
    }
    const int hk = seg / p.row_blocks, rb = seg - hk * p.row_blocks;
    int ql = p.q_lens ? p.q_lens[b] : p.Sq;
    ql = min(max(ql, 0), p.Sq);
    for (int col = warp; col < RB; col += 8) {
        const int row = rb * RB + col, i = row / p.group;
        if (row >= p.rows || i >= ql) continue;
        const int h = hk * p.group + (row - i * p.group);
        float mx = -INFINITY, sum = 0.f, o[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = 0.f;
        if (units > 0) {
            const size_t stride = (size_t)RB * (D + 2);
            for (int c = c0 + lane; c <= c1; c += 32)
                mx = fmaxf(mx, p.part[(size_t)(2 * c + (c == c0 ? 1 : 0)) * stride + RB * D + col]);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            if (mx != -INFINITY) {
#pragma unroll 4
                for (int c = c0; c <= c1; ++c) {
                    const float* slot = p.part + (size_t)(2 * c + (c == c0 ? 1 : 0)) * stride;
                    const float f = ptx::ex2(slot[RB * D + col] - mx);
                    sum = fmaf(slot[RB * (D + 1) + col], f, sum);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) o[e] = fmaf(slot[col * D + lane * kPer + e], f, o[e]);
                }
            }
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        uint16_t* dst = p.o + (((size_t)b * p.Sq + i) * p.Hq + h) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = bf16 ? ptx::pack_bf16x2(o[e] * inv, o[e + 1] * inv)
                                                         : ptx::pack_f16x2(o[e] * inv, o[e + 1] * inv);
        if (lane == 0)
            p.lse[((size_t)b * p.Hq + h) * p.Sq + i] = sum > 0.f ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
}

template <int D, int CT, int NT>
int launch_instance(bool& attr_set, const AttendParams& p, cudaStream_t stream) {
    using C = Cfg<D, CT, NT>;
    auto kernel = paged_attend_kernel<D, CT, NT>;
    if (!attr_set) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
            return ATTN_ERR_CUDA;
        attr_set = true;
    }
    kernel<<<p.ctas, C::kWarps * 32, C::kSmemBytes, stream>>>(p);
    // The merge may become resident while the attention drains; it waits for its end itself.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * p.row_blocks));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const bool bf16 = CT == kBf16 || (CT == kE4m3 && p.q_bf16);
    if (cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, C::kRows>, p, bf16) != cudaSuccess) return ATTN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int CT>
int launch_attend(bool (&attr_set)[2][3], const AttendParams& p, int D, cudaStream_t stream) {
    bool(&set)[3] = attr_set[D == 128];
    switch (block_rows(p.rows)) {
        case 8:
            return D == 128 ? launch_instance<128, CT, 1>(set[0], p, stream) : launch_instance<64, CT, 1>(set[0], p, stream);
        case 16:
            return D == 128 ? launch_instance<128, CT, 2>(set[1], p, stream) : launch_instance<64, CT, 2>(set[1], p, stream);
        default:
            return D == 128 ? launch_instance<128, CT, 4>(set[2], p, stream) : launch_instance<64, CT, 4>(set[2], p, stream);
    }
}

}  // namespace paged
}  // namespace attn
