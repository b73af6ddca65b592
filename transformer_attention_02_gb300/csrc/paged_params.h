// Host-visible parameters of the paged key/value cache's kernels (append,
// attention, merge of key ranges) and their launchers, defined in
// paged_append.cu and paged_attn_*.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "early_launch.h"

namespace attn {
namespace paged {

// Storage of the cache, with the type of the tensor-core operands it implies.
constexpr int kBf16 = 0, kF16 = 1, kE4m3 = 2;

// Device values that are out of range (page numbers, lengths, positions) set
// this bit of the device status word; what they name is left out.
constexpr unsigned int kStatusBadIndex = 2u;

constexpr int kMinScaleExp = -100;      // smallest block scale of an 8-bit cache: 2^-100

struct AppendParams {
    const uint16_t* k;            // (B, S, Hkv, D) 16-bit, `k_stride` elements from token to token
    const uint16_t* v;
    long long k_stride, v_stride;
    void* k_cache;                // (n_pages, Hkv, page, D)
    void* v_cache;
    float* k_scale;               // (n_pages, Hkv), 8-bit caches only
    float* v_scale;
    const int* block_table;       // (B, max_pages)
    const int* kv_lens;           // (B) tokens in the cache, the step's included
    const int* new_lens;          // (B) tokens of the step, or null: S
    const float* rope;            // (max_pos, D/2, {cos, sin}) or null
    int max_pos;
    int B, S, Hkv, D;
    int page_shift, max_pages, n_pages;
    int touched;                  // pages a sequence's step may touch
    int head_group;               // K/V heads a CTA takes in turn (set by the launcher)
    bool bf16;                    // type of k and v
    unsigned int* status;
};

// e4m3 or 16-bit cache by `cache`; ATTN_OK or ATTN_ERR_CUDA.
int launch_append(AppendParams p, int cache, int num_sms, cudaStream_t stream);

constexpr int kUnit = 128;        // keys of a scheduling unit

struct AttendParams {
    const uint16_t* q;            // (B, Sq, Hq, D) 16-bit, `q_stride` elements from token to token
    long long q_stride;
    const void* k_cache;          // (n_pages, Hkv, page, D)
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int* block_table;       // (B, max_pages)
    const int* kv_lens;           // (B)
    const int* q_lens;            // (B) or null: Sq
    const float* rope;            // or null
    uint16_t* o;                  // (B, Sq, Hq, D)
    float* lse;                   // (B, Hq, Sq)
    float* part;                  // 2 slots per CTA of rows x (D + 2) FP32: unnormalised O, then maxima, then sums
    int* base;                    // (B + 2) every sequence's first position in the schedule, its end, its lead
    unsigned int* status;
    float scale_log2;             // scale * log2(e)
    int max_pos;
    int B, Sq, Hq, Hkv, group;
    int rows;                     // Sq * group: query rows of a K/V head
    int row_blocks;               // ceil(rows / rows of a block)
    int page_shift, max_pages, n_pages;
    int window, sinks;            // window 0: the whole past
    int ctas;                     // grid of the attention kernel
    bool whole;                   // one CTA per segment, no parts and no merge
    bool q_bf16;                  // type of q and o (8-bit caches; 16-bit ones have q's type)
};

// Rows of a row block for `rows` query rows a K/V head: a multiple of the
// products' eight rows, at most 32.
inline int block_rows(int rows) { return rows <= 24 ? (rows <= 8 ? 8 : rows <= 16 ? 16 : 24) : 32; }

// How the attention kernel fills an SM: CTAs at once, their warps, the keys of a
// warp's stage (16 a tile) and the stages of its ring. (The reasons stand at Cfg.)
struct Plan {
    int ctas, warps, keys, stages;
};
constexpr Plan plan_of(int D, int rows_per_block, int cache) {
    const bool wide = rows_per_block > 16;
    if (cache == kE4m3) {
        if (D == 128) return !wide ? Plan{3, 4, 32, 2} : rows_per_block == 24 ? Plan{2, 4, 32, 3} : Plan{2, 4, 32, 2};
        return rows_per_block == 8 ? Plan{3, 4, 64, 2} : rows_per_block == 32 ? Plan{2, 4, 32, 3} : Plan{3, 4, 32, 3};
    }
    if (D == 128) return !wide ? Plan{2, 4, 16, 3} : Plan{1, 8, 16, 3};
    return rows_per_block == 32 ? Plan{3, 4, 16, 3} : Plan{3, 4, 32, 2};
}

// Short tables: each CTA takes one segment, with neither schedule nor merge. Up to
// three units of keys, or up to eight where the segments alone fill the device
// (1/40 of its CTAs for each unit). Measured over e4m3, 8 K/V heads of 128, one query,
// by the schedule / whole: 1 sequence of 100 keys 6.2 / 4.6 us, 250 7.0 / 5.5, 500
// 7.0 / 7.1, 1000 7.3 / 10.3; 8 sequences of 500 8.6 / 7.6, of 1000 9.8 / 10.9; 48
// of 250 10.4 / 7.6, of 1000 24.2 / 20.0.
constexpr bool takes_whole(long long segments, long long ctas, long long units) {
    return segments <= ctas && (units <= 3 || (units <= 8 && segments * 40 >= ctas * units));
}

// The attention and the merge of its parts, for one cache type CT (kBf16,
// kF16, kE4m3). attr_set caches, per context and instance [D is 128][rows of a
// block 8, 16, 24, 32], that the shared-memory attribute has been set.
template <int CT>
int launch_attend(bool (&attr_set)[2][4], const AttendParams& p, int D, cudaStream_t stream);

// An attention goes by the gathered pages (paged_gather.cu) from kChunkRows
// queries a sequence and kChunkTiles tiles of 256 rows of a head: a third of the
// SMs. Measured over e4m3, 32/8 heads of 128, by the cache itself / gathered: 16
// sequences of 8192 keys, 128 queries 850 / 514 us, 256 queries 1675 / 566; two,
// 128 queries (64 tiles, half filled) 121 / 116; one sequence of 32768 keys, 128
// queries (32 tiles) 215 / 406.
constexpr int kChunkRows = 128;
constexpr int kChunkTiles = 48;
constexpr long long kChunkLimit = 4LL << 30;     // bytes of gathered tensors at most

struct GatherParams {
    const void* k_cache;          // (n_pages, Hkv, page, D)
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int* block_table;
    const int* kv_lens;
    const int* q_lens;            // or null
    uint16_t* k_out;              // (B, cap, Hkv, D)
    uint16_t* v_out;
    const uint16_t* q;            // (B, Sq, Hq, D), `q_stride` elements from token to token
    long long q_stride;
    uint16_t* q_out;              // (B, Sq, Hq, D), with a table only
    const float* rope;            // or null: the queries are read where they are
    int max_pos;
    int B, Sq, Hq, Hkv, D;
    int cap;                      // keys a sequence: max_pages * page
    int page_shift, max_pages, n_pages;
    int window, sinks;
    long long copies;             // CTAs that gather (set by the launcher)
    bool bf16;
    unsigned int* status;
};

int launch_gather(GatherParams p, int cache, cudaStream_t stream);

}  // namespace paged
}  // namespace attn
