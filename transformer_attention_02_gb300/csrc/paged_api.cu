// Entry points of the paged key/value cache (declared in include/attn.h):
// argument checks, workspace layout and launches of the append and of the
// attention over the cache.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "attn_launch.h"
#include "paged_params.h"

namespace {

using namespace attn;

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

constexpr size_t kWorkspaceAlign = 256;
size_t align_up(size_t x) { return (x + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign; }

// Sizes the append and the attention share. A page holds a power of two of
// tokens, 16 to 256; every product that indexes memory fits its type.
int check_cache(int B, int S, int Hkv, int D, int page, int max_pages, int n_pages, int cache) {
    if (B < 0 || S < 0 || Hkv <= 0 || D <= 0 || max_pages <= 0 || n_pages <= 0) return ATTN_ERR_INVALID_ARG;
    if (cache != ATTN_CACHE_16BIT && cache != ATTN_CACHE_E4M3) return ATTN_ERR_INVALID_ARG;
    if (page < 16 || page > 256 || (page & (page - 1)) != 0) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_pages * page > (1 << 30) || S > (1 << 30)) return ATTN_ERR_INVALID_ARG;
    if ((long long)Hkv * page * D > (1 << 30)) return ATTN_ERR_INVALID_ARG;          // bytes of a page in 32 bits
    return ATTN_OK;
}

bool rope_ok(const float* table, int max_pos) { return !table || (aligned(table, 16) && max_pos > 0); }

int page_shift_of(int page) {
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

int kv_append_impl(const void* k, const void* v, long long k_stride, long long v_stride, void* k_cache, void* v_cache,
                   float* k_scale, float* v_scale, const int* block_table, const int* kv_lens, const int* new_lens,
                   int B, int S, int Hkv, int D, int page, int max_pages, int n_pages, int cache,
                   const float* rope_table, int max_pos, cudaStream_t stream, bool bf16) {
    int rc = check_cache(B, S, Hkv, D, page, max_pages, n_pages, cache);
    if (rc != ATTN_OK) return rc;
    if (B == 0 || S == 0) return ATTN_OK;
    if (!k || !v || !k_cache || !v_cache || !block_table || !kv_lens) return ATTN_ERR_INVALID_ARG;
    const bool e4m3 = cache == ATTN_CACHE_E4M3;
    if (e4m3 && (!k_scale || !v_scale)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(new_lens, 4))
        return ATTN_ERR_INVALID_ARG;
    if (k_stride < (long long)Hkv * D || v_stride < (long long)Hkv * D || k_stride % 8 != 0 || v_stride % 8 != 0)
        return ATTN_ERR_INVALID_ARG;
    if (!rope_ok(rope_table, max_pos)) return ATTN_ERR_INVALID_ARG;
    const int touched = (int)std::min<long long>(max_pages, ((long long)S + page - 2) / page + 1);
    if ((long long)B * touched * Hkv * 2 > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;

    DeviceState dev{};
    rc = device_state(&dev);
    if (rc != ATTN_OK) return rc;
    paged::AppendParams p{};
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.new_lens = new_lens;
    p.rope = rope_table;
    p.max_pos = max_pos;
    p.B = B;
    p.S = S;
    p.Hkv = Hkv;
    p.D = D;
    p.page_shift = page_shift_of(page);
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.touched = touched;
    p.bf16 = bf16;
    p.status = dev.status;
    return paged::launch_append(p, e4m3 ? paged::kE4m3 : bf16 ? paged::kBf16 : paged::kF16, dev.num_sms, stream);
}

// A segment's units in the schedule at most: its keys, one unit more for the
// sinks, and its lead.
long long span_bound(long long max_keys) { return (max_keys + paged::kUnit - 1) / paged::kUnit + 4; }

// CTAs of the attention: as many as the device holds at once, or as the longest
// lists could give work to (max_keys 0: any length).
int attend_ctas(int B, int Hkv, int rows, int D, int cache, long long max_keys, int sms) {
    const int rb = paged::block_rows(rows);
    const long long all = (long long)sms * paged::plan_of(D, rb, cache).ctas;
    if (max_keys <= 0) return (int)all;
    const long long segments = (long long)B * Hkv * ((rows + rb - 1) / rb);
    return (int)std::min(all, segments > all ? all : segments * span_bound(max_keys));
}

// Workspace of the attention: the place of every sequence in the schedule, then
// two FP32 parts (unnormalised O, maximum, sum) for each CTA.
size_t attend_workspace(int B, int rows, int D, int ctas, size_t* part_off) {
    *part_off = align_up((size_t)(B + 2) * sizeof(int));
    return *part_off + (size_t)ctas * 2 * paged::block_rows(rows) * (D + 2) * sizeof(float);
}

// Workspace of a long chunk: gathered keys and values, then rotated queries.
struct ChunkLayout {
    int cap = 0;                       // keys a sequence
    size_t v_off = 0, q_off = 0, total = 0;
};

// False where the gathered path does not apply (few queries or tiles, or too large).
bool chunk_layout(int B, int Hq, int Hkv, int Sq, int D, long long max_keys, ChunkLayout* c) {
    if (Sq < paged::kChunkRows || max_keys <= 0) return false;
    if ((long long)B * Hq * ((Sq + 255) / 256) < paged::kChunkTiles) return false;
    c->cap = (int)max_keys;
    const double kv = 2.0 * B * c->cap * Hkv * D, q = 2.0 * B * Sq * Hq * D;
    if (2 * kv + q > (double)paged::kChunkLimit || (double)B * (c->cap / 128 + 1) * Hkv + q / 16 / 256 > 2e9) return false;
    c->v_off = align_up((size_t)kv);
    c->q_off = 2 * c->v_off;
    c->total = c->q_off + align_up((size_t)q);
    return true;
}

int attend_impl(const void* q, long long q_stride, const void* k_cache, const void* v_cache, const float* k_scale,
                const float* v_scale, const int* block_table, const int* kv_lens, const int* q_lens, void* o, float* lse,
                int B, int Hq, int Hkv, int Sq, int D, int page, int max_pages, int n_pages, int cache, float scale,
                int window, int sinks, const float* rope_table, int max_pos, void* workspace, size_t workspace_bytes,
                cudaStream_t stream, bool bf16) {
    int rc = check_cache(B, Sq, Hkv, D, page, max_pages, n_pages, cache);
    if (rc != ATTN_OK) return rc;
    if (Hq < 0 || Hq % Hkv != 0 || window < 0 || sinks < 0) return ATTN_ERR_INVALID_ARG;
    if (B == 0 || Sq == 0 || Hq == 0) return ATTN_OK;
    if (!q || !k_cache || !v_cache || !block_table || !kv_lens || !o || !lse) return ATTN_ERR_INVALID_ARG;
    const bool e4m3 = cache == ATTN_CACHE_E4M3;
    if (e4m3 && (!k_scale || !v_scale)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(lse, 4) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(kv_lens, 4) ||
        !aligned(q_lens, 4))
        return ATTN_ERR_INVALID_ARG;
    if (q_stride < (long long)Hq * D || q_stride % 8 != 0) return ATTN_ERR_INVALID_ARG;
    if (!rope_ok(rope_table, max_pos)) return ATTN_ERR_INVALID_ARG;
    const long long rows = (long long)Sq * (Hq / Hkv);
    if (rows > (1 << 30)) return ATTN_ERR_INVALID_ARG;
    const int rb = paged::block_rows((int)rows);
    const long long row_blocks = (rows + rb - 1) / rb;
    const long long max_keys = (long long)max_pages * page;
    if ((long long)B * Hkv * row_blocks > 0x7fffffffLL / span_bound(max_keys)) return ATTN_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, kWorkspaceAlign)) return ATTN_ERR_INVALID_ARG;
    size_t part_off = 0;
    ChunkLayout chunk;
    const bool gathered = chunk_layout(B, Hq, Hkv, Sq, D, max_keys, &chunk) && workspace_bytes >= chunk.total;
    const int type = e4m3 ? paged::kE4m3 : bf16 ? paged::kBf16 : paged::kF16;
    const int ctas = attend_ctas(B, Hkv, (int)rows, D, type, max_keys, device_sm_count());
    if (!gathered && workspace_bytes < attend_workspace(B, (int)rows, D, ctas, &part_off)) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt((float)D);
    constexpr int kAllKeys = 1 << 30;                     // a longer window hides nothing; differences stay in 32 bits
    window = std::min(window, kAllKeys);

    DeviceState dev{};
    rc = device_state(&dev);
    if (rc != ATTN_OK) return rc;
    if (gathered) {
        char* const ws = static_cast<char*>(workspace);
        paged::GatherParams g{};
        g.k_cache = k_cache;
        g.v_cache = v_cache;
        g.k_scale = k_scale;
        g.v_scale = v_scale;
        g.block_table = block_table;
        g.kv_lens = kv_lens;
        g.q_lens = q_lens;
        g.k_out = reinterpret_cast<uint16_t*>(ws);
        g.v_out = reinterpret_cast<uint16_t*>(ws + chunk.v_off);
        g.q = static_cast<const uint16_t*>(q);
        g.q_stride = q_stride;
        g.q_out = reinterpret_cast<uint16_t*>(ws + chunk.q_off);
        g.rope = rope_table;
        g.max_pos = max_pos;
        g.B = B;
        g.Sq = Sq;
        g.Hq = Hq;
        g.Hkv = Hkv;
        g.D = D;
        g.cap = chunk.cap;
        g.page_shift = page_shift_of(page);
        g.max_pages = max_pages;
        g.n_pages = n_pages;
        g.window = window;
        g.sinks = sinks;
        g.bf16 = bf16;
        g.status = dev.status;
        rc = paged::launch_gather(g, type, stream);
        if (rc != ATTN_OK) return rc;
        return launch_ragged(rope_table ? g.q_out : q, rope_table ? (long long)Hq * D : q_stride, g.k_out, g.v_out, o, lse, B,
                             Hq, Hkv, Sq, chunk.cap, D, scale, window > 0 ? window : kAllKeys,
                             window > 0 ? sinks : 0, kv_lens, q_lens, block_table, page_shift_of(page), n_pages, stream,
                             bf16);
    }
    paged::AttendParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride = q_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.q_lens = q_lens;
    p.rope = rope_table;
    p.o = static_cast<uint16_t*>(o);
    p.lse = lse;
    p.base = static_cast<int*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + part_off);
    p.status = dev.status;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.max_pos = max_pos;
    p.B = B;
    p.Sq = Sq;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.rows = (int)rows;
    p.row_blocks = (int)row_blocks;
    p.page_shift = page_shift_of(page);
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.window = window;
    p.sinks = sinks;
    const long long segments = (long long)B * Hkv * row_blocks;
    p.whole = paged::takes_whole(segments, (long long)dev.num_sms * paged::plan_of(D, rb, type).ctas,
                                 (max_keys + paged::kUnit - 1) / paged::kUnit);
    p.ctas = p.whole ? (int)segments : ctas;
    p.q_bf16 = bf16;
    if (e4m3) return paged::launch_attend<paged::kE4m3>(dev.paged_attr_set[paged::kE4m3], p, D, stream);
    return bf16 ? paged::launch_attend<paged::kBf16>(dev.paged_attr_set[paged::kBf16], p, D, stream)
                : paged::launch_attend<paged::kF16>(dev.paged_attr_set[paged::kF16], p, D, stream);
}

}  // namespace

extern "C" {

int attn_kv_append(const void* k, const void* v, long long k_stride, long long v_stride, void* k_cache, void* v_cache,
                   float* k_scale, float* v_scale, const int* block_table, const int* kv_lens, const int* new_lens,
                   int B, int S, int Hkv, int D, int page, int max_pages, int n_pages, int cache_kind,
                   const float* rope_table, int max_pos, attn_stream_t stream) {
    return kv_append_impl(k, v, k_stride, v_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, new_lens, B,
                          S, Hkv, D, page, max_pages, n_pages, cache_kind, rope_table, max_pos,
                          reinterpret_cast<cudaStream_t>(stream), true);
}

int attn_kv_append_f16(const void* k, const void* v, long long k_stride, long long v_stride, void* k_cache,
                       void* v_cache, float* k_scale, float* v_scale, const int* block_table, const int* kv_lens,
                       const int* new_lens, int B, int S, int Hkv, int D, int page, int max_pages, int n_pages,
                       int cache_kind, const float* rope_table, int max_pos, attn_stream_t stream) {
    return kv_append_impl(k, v, k_stride, v_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, new_lens, B,
                          S, Hkv, D, page, max_pages, n_pages, cache_kind, rope_table, max_pos,
                          reinterpret_cast<cudaStream_t>(stream), false);
}

size_t attn_paged_workspace_bytes(int B, int Hq, int Hkv, int Sq, int D, long long max_keys) {
    if (max_keys < 0 || max_keys > (1 << 30) || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Sq <= 0 || (D != 64 && D != 128)) return 0;
    if ((long long)Sq * (Hq / Hkv) > (1 << 30)) return 0;
    size_t part_off = 0;
    const int rows = Sq * (Hq / Hkv);
    ChunkLayout chunk;
    if (chunk_layout(B, Hq, Hkv, Sq, D, max_keys, &chunk)) return chunk.total;
    // (enough for either kind of cache)
    const int sms = device_sm_count(), ctas = std::max(attend_ctas(B, Hkv, rows, D, paged::kE4m3, max_keys, sms),
                                                       attend_ctas(B, Hkv, rows, D, paged::kBf16, max_keys, sms));
    return attend_workspace(B, rows, D, ctas, &part_off);
}

int attn_fwd_paged(const void* q, long long q_stride, const void* k_cache, const void* v_cache, const float* k_scale,
                   const float* v_scale, const int* block_table, const int* kv_lens, const int* q_lens, void* o,
                   float* lse, int B, int Hq, int Hkv, int Sq, int D, int page, int max_pages, int n_pages,
                   int cache_kind, float scale, int window, int sinks, const float* rope_table, int max_pos,
                   void* workspace, size_t workspace_bytes, attn_stream_t stream) {
    return attend_impl(q, q_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_lens, o, lse, B, Hq, Hkv,
                       Sq, D, page, max_pages, n_pages, cache_kind, scale, window, sinks, rope_table, max_pos, workspace,
                       workspace_bytes, reinterpret_cast<cudaStream_t>(stream), true);
}

int attn_fwd_paged_f16(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                       const float* k_scale, const float* v_scale, const int* block_table, const int* kv_lens,
                       const int* q_lens, void* o, float* lse, int B, int Hq, int Hkv, int Sq, int D, int page,
                       int max_pages, int n_pages, int cache_kind, float scale, int window, int sinks,
                       const float* rope_table, int max_pos, void* workspace, size_t workspace_bytes,
                       attn_stream_t stream) {
    return attend_impl(q, q_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_lens, o, lse, B, Hq, Hkv,
                       Sq, D, page, max_pages, n_pages, cache_kind, scale, window, sinks, rope_table, max_pos, workspace,
                       workspace_bytes, reinterpret_cast<cudaStream_t>(stream), false);
}

}  // extern "C"
