// Entry points of the attention's backward pass (declared in include/attn.h):
// argument checks, workspace layout and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "attn_launch.h"
#include "bwd_params.h"
#include "checkpoint_params.h"

namespace {

using namespace attn;

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

constexpr size_t kWorkspaceAlign = 256;
size_t align_up(size_t x) { return (x + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign; }

bool is_additive(int mask_kind) { return mask_kind == ATTN_MASK_ADDITIVE || mask_kind == ATTN_MASK_CAUSAL_ADDITIVE; }

// Where there are few tiles their walks are cut into parts, as many as an estimate finds the quickest, in blocks of 128 x 128
// pairs: a part costs its blocks and kTileCost for its beginning and end; walks of one length run in waves of the device's
// SMs, those of several lengths (under a causal mask, or with the sinks of a window) fill each other's gaps, so that the
// longest part or an SM's share of everything bounds them; joining costs a launch and two passes over the sums. The keys of a
// window's sinks are seen by all queries: with many tiles the walks of theirs alone are cut. Measured, bf16 heads of 128, whole
// and cut: 4096 causal tokens of 8 heads on one K/V head 382 and 125 us, 1024 of 32 heads on one 362 and 79, 16384 of one head
// 301 and 191, 128 queries of 8 heads over 16384 keys 182 and 75; with 4 sinks, window 128 over
// 16384 tokens of 32 / 8 heads 1084 and 389, over 32768 of 16 heads of 64 on two 3328 and 330 (238 without sinks).
constexpr int kPartBlocks = 4, kMaxParts = 64;      // a part of the longest walk has no fewer blocks
constexpr int kSinkTiles = 2;                       // parts of the sinks' tiles, for each SM, at most
constexpr double kTileCost = 3.0, kJoinCost = 2.0, kSumCost = 0.04;
struct Walks {
    double cut, longest;            // walks that may be cut, the longest of them
    double tiles, other;            // all walks, the longest of those that stay whole
    double total;                   // blocks of all walks together
    bool even;                      // of one length
};
struct Choice {
    int parts;
    double cost;
};
Choice parts_of(const Walks& w, int sms, int most) {
    Choice best{1, 0.0};
    for (int s = 1; s <= most && (s == 1 || s <= w.longest / kPartBlocks); ++s) {
        double cost = w.even ? std::ceil(w.cut * s / sms) * (std::ceil(w.longest / s) + kTileCost)
                             : std::max(std::max(w.longest / s, w.other) + kTileCost,
                                        (w.total + kTileCost * (w.tiles + w.cut * (s - 1))) / sms);
        if (s > 1) cost += kJoinCost + kSumCost * w.cut * s;
        if (s == 1 || cost < best.cost) best = {s, cost};
    }
    return best;
}
// All walks are cut, or none. (With as many tiles as these nothing is won.)
Choice parts_of_all(double tiles, double longest, double total, bool even, int sms, int most = kMaxParts) {
    return parts_of({tiles, longest, tiles, 0.0, total, even}, sms, tiles >= 4.0 * sms ? 1 : most);
}
struct Parts {
    int dq = 1, dkv = 1;
    int sink_kb = 0;                // key blocks of the sinks, where theirs alone are cut
    size_t bytes = 0;               // of the larger of the two sets of sums: they are used one after the other
};
// Parts at most of each of the `kb` tiles of sinks that every K/V head has.
int most_sink_parts(double heads, double kb, double walk, int sms) {
    return (int)std::min({(double)kMaxParts, std::floor(walk / kPartBlocks), std::floor(kSinkTiles * sms / (heads * kb))});
}
Parts parts_for(int B, int Hq, int Hkv, int Sq, int Sk, int D, int mask_kind) {
    const int sms = device_sm_count();
    const double nq = (double)(bwd::padded_rows(Sq) / bwd::kBlock), nk = (double)(bwd::padded_rows(Sk) / bwd::kBlock);
    const double q_tiles = B * (double)Hq * nq, kv_tiles = B * (double)Hkv * nk, kv_walk = nq * (Hq / Hkv);
    Parts s;
    const bool triangle = mask_kind == ATTN_MASK_CAUSAL || mask_kind == ATTN_MASK_CAUSAL_ADDITIVE;
    const double share = triangle ? 0.5 : 1.0;
    if (!is_additive(mask_kind)) s.dq = parts_of_all(q_tiles, nk, share * q_tiles * nk, !triangle, sms).parts;
    s.dkv = parts_of_all(kv_tiles, kv_walk, share * kv_tiles * kv_walk, !triangle, sms).parts;
    const size_t vectors = (size_t)D * sizeof(float);
    const size_t q = s.dq > 1 ? s.dq * vectors * B * Sq * Hq : 0, kv = s.dkv > 1 ? s.dkv * vectors * 2 * B * Sk * Hkv : 0;
    // (of all sinks that a window may have: kb * most_sink_parts(.., kb, ..) tiles a head)
    const double heads = B * (double)Hkv;
    const double most = std::min(nk * std::min((double)kMaxParts, std::floor(kv_walk / kPartBlocks)), kSinkTiles * sms / heads);
    const size_t sinks = mask_kind == ATTN_MASK_CAUSAL ? (size_t)(most * heads) * 2 * bwd::kBlock * vectors : 0;
    s.bytes = align_up(std::max({q, kv, sinks}));
    return s;
}
// With a window: all walks in no more parts than without, for which the workspace is, or the sinks' in as many as that holds.
Parts parts_in_window(Parts s, int B, int Hq, int Hkv, int Sq, int Sk, int window, int sinks) {
    const int sms = device_sm_count();
    const double nq = (double)(bwd::padded_rows(Sq) / bwd::kBlock), nk = (double)(bwd::padded_rows(Sk) / bwd::kBlock);
    const double seen = std::floor(((double)window + bwd::kBlock - 2) / bwd::kBlock) + 1;      // blocks that touch a tile's windows
    const double sink_kb = std::min(nk, std::ceil((double)sinks / bwd::kBlock));
    const double q_tiles = B * (double)Hq * nq, q_walk = std::min(nk, seen + sink_kb);
    const double heads = B * (double)Hkv, G = Hq / Hkv, kv_walk = std::min(nq, seen) * G;
    s.dq = parts_of_all(q_tiles, q_walk, q_tiles * q_walk, true, sms, s.dq).parts;
    const double total = heads * ((nk - sink_kb) * kv_walk + sink_kb * nq * G);
    const Choice all = parts_of_all(heads * nk, sink_kb > 0 ? nq * G : kv_walk, total, sink_kb == 0, sms, s.dkv);
    s.dkv = all.parts;
    if (sink_kb > 0 && sink_kb < nk) {
        const Choice sink = parts_of({heads * sink_kb, nq * G, heads * nk, kv_walk, total, false}, sms,
                                     std::max(1, most_sink_parts(heads, sink_kb, nq * G, sms)));
        if (sink.parts > 1 && sink.cost < all.cost) {
            s.dkv = sink.parts;
            s.sink_kb = (int)sink_kb;
        }
    }
    return s;
}

// The head: two tile counters, and behind 32 bytes the words of fp16's ranges, one for each part of a (b, K/V head). Then three
// statistics for every query row, the third with an additive mask only.
constexpr size_t kHead = 1024, kCounters = 8;       // bytes at least; words

// Neighbouring K/V heads of a block (2^shift) and parts of each in fp16's pass over dO and V: two blocks an SM. More heads are
// quicker, but a tile's warps read a head's parts at once where those are 32 at most. No part has less than a block's four vectors
// a row of lanes.
struct RangeSplit {
    int shift, parts;
};
RangeSplit range_split(int B, int Hq, int Hkv, int Sq, int Sk, int D) {
    const long long heads = (long long)B * Hkv, blocks = 2LL * device_sm_count();
    RangeSplit s{0, 1};
    while (s.shift < 3 && Hkv % (2 << s.shift) == 0 && (heads >> (s.shift + 1)) * 32 >= blocks) ++s.shift;
    const long long rows = (long long)Sq * (Hq / Hkv) + Sk, each = 4 * (bwd::kRangeThreads / (D / 8) >> s.shift);
    s.parts = (int)std::min({std::max(1LL, blocks / (heads >> s.shift)), (rows + each - 1) / each, 160LL});
    return s;
}
size_t head_bytes(int B, int Hq, int Hkv, int Sq, int Sk, int D) {
    const size_t words = kCounters + (size_t)B * Hkv * range_split(B, Hq, Hkv, Sq, Sk, D).parts;
    return std::max(kHead, align_up(words * sizeof(unsigned int)));
}
size_t stat_bytes(int B, int Hq, int Sq) { return align_up((size_t)B * Hq * bwd::padded_rows(Sq) * sizeof(float)); }
size_t bwd_workspace(int B, int Hq, int Hkv, int Sq, int Sk, int D, int mask_kind) {
    return head_bytes(B, Hq, Hkv, Sq, Sk, D) + stat_bytes(B, Hq, Sq) * (is_additive(mask_kind) ? 3 : 2) +
           parts_for(B, Hq, Hkv, Sq, Sk, D, mask_kind).bytes;
}

// A tensor of tokens: pointer, distance of tokens, H * D values a token. Null only where it is empty.
bool tokens_ok(const void* ptr, long long stride, int B, int S, int H, int D) {
    if ((long long)B * S * H == 0) return true;
    // (the distances of a tensor map have 40 bits)
    return ptr && aligned(ptr, 16) && stride >= (long long)H * D && stride % 8 == 0 && stride < (1LL << 39) / std::max(1, S);
}

// Whether one of the first `written` of these tensors begins where another of them does (null: no tensor).
template <int N>
bool any_begins_in(const void* const (&all)[N], int written) {
    for (int i = 0; i < written; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && all[i] && all[i] == all[j]) return true;
    return false;
}

int check_sizes(int B, int Hq, int Hkv, int Sq, int Sk, int D) {
    if (B < 0 || Hq < 0 || Hkv <= 0 || Sq < 0 || Sk < 0 || D <= 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (Sq > (1 << 30) || Sk > (1 << 30)) return ATTN_ERR_INVALID_ARG;
    const long long nq = bwd::padded_rows(Sq) / bwd::kBlock, nk = bwd::padded_rows(Sk) / bwd::kBlock;
    if ((double)B * Hq * nq > 2147483647.0 || (double)B * Hkv * nk > 2147483647.0 || (double)nq * (Hq / Hkv) > 2147483647.0)
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

int zero_tokens(void* ptr, long long stride, int B, int S, int H, int D, cudaStream_t stream) {
    if ((long long)B * S * H == 0) return ATTN_OK;
    return cudaMemset2DAsync(ptr, (size_t)stride * 2, 0, (size_t)H * D * 2, (size_t)B * S, stream) == cudaSuccess
               ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, bool BF16, bool ADDITIVE>
int launch_both(const DeviceState& dev, const CUtensorMap* maps, bwd::BwdParams& p, unsigned int* counters, const Parts& parts,
                cudaStream_t stream) {
    bool (*attr)[2] = dev.bwd_attr_set[D == 128][BF16][ADDITIVE];
    const int dq_tiles = p.B * p.Hq * p.n_qb * parts.dq;
    p.cut = p.B * p.Hkv * (parts.sink_kb ? parts.sink_kb : p.n_kb);
    p.part_rows = parts.sink_kb ? parts.sink_kb * bwd::kBlock : p.Sk;
    const int dkv_tiles = p.B * p.Hkv * p.n_kb + p.cut * (parts.dkv - 1);
    int rc;
    // Where every tile has a CTA of its own, what the counters hold is of no account (100 tokens of 8 heads: 17.3 us with them set, 16.3 without).
    if (BF16 && std::max(dq_tiles, dkv_tiles) > dev.num_sms && (rc = bwd::launch_begin(counters, stream)) != ATTN_OK) return rc;
    p.splits = parts.dq;
    p.n_tiles = dq_tiles;
    p.counter = counters;
    rc = bwd::launch_dq<D, BF16, ADDITIVE>(attr[0], maps[0], maps[1], maps[2], maps[3], p,
                                               std::min(p.n_tiles, dev.num_sms), stream);
    if (rc != ATTN_OK) return rc;
    if (p.splits > 1) {
        bwd::JoinParams j{};
        j.part = p.part;
        j.apart = (long long)p.B * p.Sq * p.Hq * D;
        j.splits = p.splits;
        j.out = static_cast<uint16_t*>(p.dq);
        j.tokens = (long long)p.B * p.Sq;
        j.rows = j.out_rows = p.Sq;
        j.stride = p.dq_stride;
        j.width = p.Hq * D;
        j.factor = p.scale;
        if ((rc = bwd::launch_join(&j, 1, BF16, dev.num_sms, stream)) != ATTN_OK) return rc;
    }
    p.splits = parts.dkv;
    p.n_tiles = dkv_tiles;
    p.counter = counters + 1;
    rc = bwd::launch_dkv<D, BF16, ADDITIVE>(attr[1], maps[0], maps[1], maps[2], maps[3], p, std::min(p.n_tiles, dev.num_sms), stream);
    if (rc != ATTN_OK || p.splits == 1) return rc;
    bwd::JoinParams j[2] = {};
    for (int i = 0; i < 2; ++i) {                                 // dV, dK
        const long long plane = (long long)p.B * p.part_rows * p.Hkv * D;
        j[i].part = p.part + i * plane;
        j[i].apart = 2 * plane;
        j[i].splits = p.splits;
        j[i].out = static_cast<uint16_t*>(i ? p.dk : p.dv);
        j[i].tokens = (long long)p.B * p.part_rows;
        j[i].rows = p.part_rows;
        j[i].out_rows = p.Sk;
        j[i].stride = i ? p.dk_stride : p.dv_stride;
        j[i].width = p.Hkv * D;
        j[i].factor = i ? p.scale : 1.f;
    }
    return bwd::launch_join(j, 2, BF16, dev.num_sms, stream);
}

int bwd_impl(const void* d_o, const void* q, const void* k, const void* v, const void* o, const float* lse, void* dq,
             void* dk, void* dv, long long q_stride, long long k_stride, long long v_stride, long long dq_stride,
             long long dk_stride, long long dv_stride, int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
             int mask_kind, const float* mask, int window, int sinks, void* workspace, size_t workspace_bytes,
             cudaStream_t stream, bool bf16, bool check_only = false) {
    int rc = check_sizes(B, Hq, Hkv, Sq, Sk, D);
    if (rc != ATTN_OK) return rc;
    if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_CAUSAL_ADDITIVE || window < 0 || sinks < 0)
        return ATTN_ERR_INVALID_ARG;
    if (window > 0 && mask_kind != ATTN_MASK_CAUSAL) return ATTN_ERR_INVALID_ARG;
    const long long q_values = (long long)B * Sq * Hq, kv_values = (long long)B * Sk;
    if (!tokens_ok(q, q_stride, B, Sq, Hq, D) || !tokens_ok(k, k_stride, B, Sk, Hkv, D) ||
        !tokens_ok(v, v_stride, B, Sk, Hkv, D) || !tokens_ok(dq, dq_stride, B, Sq, Hq, D) ||
        !tokens_ok(dk, dk_stride, B, Sk, Hkv, D) || !tokens_ok(dv, dv_stride, B, Sk, Hkv, D) ||
        !tokens_ok(d_o, (long long)Hq * D, B, Sq, Hq, D) || !tokens_ok(o, (long long)Hq * D, B, Sq, Hq, D))
        return ATTN_ERR_INVALID_ARG;
    if (q_values > 0 && kv_values > 0) {                          // what is written begins where another tensor does
        const void* const all[] = {dq, dk, dv, workspace, d_o, q, k, v, o, lse, mask};
        if (any_begins_in(all, 4)) return ATTN_ERR_INVALID_ARG;
    }
    const bool additive = is_additive(mask_kind);
    if (q_values > 0 && (!lse || !aligned(lse, 4))) return ATTN_ERR_INVALID_ARG;
    if (additive && q_values > 0 && kv_values > 0 && (!mask || !aligned(mask, 4))) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt((float)D);
    if (q_values == 0 || kv_values == 0) {                        // no pair of a query and a key: no gradients
        if (q_values == 0 && kv_values == 0) return ATTN_OK;
        DeviceState dev{};
        if ((rc = device_state(&dev)) != ATTN_OK || (rc = zero_tokens(dq, dq_stride, B, Sq, Hq, D, stream)) != ATTN_OK ||
            (rc = zero_tokens(dk, dk_stride, B, Sk, Hkv, D, stream)) != ATTN_OK)
            return rc;
        return zero_tokens(dv, dv_stride, B, Sk, Hkv, D, stream);
    }
    if (!workspace || !aligned(workspace, kWorkspaceAlign) || workspace_bytes < bwd_workspace(B, Hq, Hkv, Sq, Sk, D, mask_kind))
        return ATTN_ERR_INVALID_ARG;
    if (check_only) return ATTN_OK;

    DeviceState dev{};
    rc = device_state(&dev);
    if (rc != ATTN_OK) return rc;
    CUtensorMap maps[4];
    if (encode_tokens(&maps[0], q, B, Sq, Hq, D, bf16, q_stride) != ATTN_OK ||
        encode_tokens(&maps[1], k, B, Sk, Hkv, D, bf16, k_stride) != ATTN_OK ||
        encode_tokens(&maps[2], v, B, Sk, Hkv, D, bf16, v_stride) != ATTN_OK ||
        encode_tokens(&maps[3], d_o, B, Sq, Hq, D, bf16, (long long)Hq * D) != ATTN_OK)
        return ATTN_ERR_CUDA;
    const size_t stat = stat_bytes(B, Hq, Sq);
    unsigned int* const counters = static_cast<unsigned int*>(workspace);
    char* const ws = static_cast<char*>(workspace) + head_bytes(B, Hq, Hkv, Sq, Sk, D);

    Parts parts = parts_for(B, Hq, Hkv, Sq, Sk, D, mask_kind);
    if (window > 0) parts = parts_in_window(parts, B, Hq, Hkv, Sq, Sk, window, sinks);

    constexpr int kAllKeys = 1 << 30;                     // a longer window hides nothing; differences stay in 32 bits
    bwd::BwdParams p{};
    if (!bf16) {
        bwd::RangeParams r{};
        r.counters = counters;
        r.range = counters + kCounters;
        r.d_o = static_cast<const uint16_t*>(d_o);
        r.v = static_cast<const uint16_t*>(v);
        r.v_stride = v_stride;
        const RangeSplit split = range_split(B, Hq, Hkv, Sq, Sk, D);
        r.shift = split.shift;
        r.parts = split.parts;
        r.units = (B * Hkv >> r.shift) * r.parts;                 // (parts where they are few)
        r.Hkv = Hkv;
        r.group = Hq / Hkv;
        r.Sq = Sq;
        r.Sk = Sk;
        p.range = r.range;
        p.n_range = r.parts;
        rc = bwd::launch_range(r, D, dev.num_sms, stream);
        if (rc != ATTN_OK) return rc;
    }
    p.o = static_cast<const uint16_t*>(o);
    p.lse = lse;
    p.neg_lse = reinterpret_cast<float*>(ws);
    p.neg_delta = reinterpret_cast<float*>(ws + stat);
    p.inv_sum = additive ? reinterpret_cast<float*>(ws + 2 * stat) : nullptr;
    p.part = reinterpret_cast<float*>(ws + (additive ? 3 : 2) * stat);
    p.mask = additive ? mask : nullptr;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dq_stride = dq_stride;
    p.dk_stride = dk_stride;
    p.dv_stride = dv_stride;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.Sq = Sq;
    p.Sk = Sk;
    p.Sp = (int)bwd::padded_rows(Sq);
    p.group = Hq / Hkv;
    p.n_qb = p.Sp / bwd::kBlock;
    p.n_kb = (int)(bwd::padded_rows(Sk) / bwd::kBlock);
    p.off = Sk - Sq;
    p.causal = mask_kind == ATTN_MASK_CAUSAL || mask_kind == ATTN_MASK_CAUSAL_ADDITIVE;
    p.window = std::min(window, kAllKeys);
    p.sinks = window > 0 ? std::min(sinks, kAllKeys) : 0;
    p.sink_kb = std::min(p.n_kb, (p.sinks + bwd::kBlock - 1) / bwd::kBlock);
    p.vec8 = aligned(dq, 32) && aligned(dk, 32) && aligned(dv, 32) && dq_stride % 16 == 0 && dk_stride % 16 == 0 &&
             dv_stride % 16 == 0;
    p.stall = dev.stall;
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = dev.timeout_ns;
    p.status = dev.status;
    if (D == 128) {
        if (additive) return bf16 ? launch_both<128, true, true>(dev, maps, p, counters, parts, stream) : launch_both<128, false, true>(dev, maps, p, counters, parts, stream);
        return bf16 ? launch_both<128, true, false>(dev, maps, p, counters, parts, stream) : launch_both<128, false, false>(dev, maps, p, counters, parts, stream);
    }
    if (additive) return bf16 ? launch_both<64, true, true>(dev, maps, p, counters, parts, stream) : launch_both<64, false, true>(dev, maps, p, counters, parts, stream);
    return bf16 ? launch_both<64, true, false>(dev, maps, p, counters, parts, stream) : launch_both<64, false, false>(dev, maps, p, counters, parts, stream);
}

// ----------------------------------------------------- 8-bit checkpoints

int check_vectors(const void* x, long long stride, const void* codes, const float* scale, int B, int S, int H, int D) {
    if (B < 0 || S < 0 || H < 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if ((double)B * S * H > (double)(1LL << 48)) return ATTN_ERR_INVALID_ARG;
    if ((long long)B * S * H == 0) return ATTN_OK;
    if (!x || !codes || !scale || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return ATTN_ERR_INVALID_ARG;
    return stride >= (long long)H * D && stride % 8 == 0 ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

checkpoint::Tensor vectors_of(const void* x, long long stride, const void* codes, const float* scale, int B, int S, int H) {
    checkpoint::Tensor t;
    t.x = static_cast<uint16_t*>(const_cast<void*>(x));
    t.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    t.scale = const_cast<float*>(scale);
    t.stride = stride;
    t.tokens = (long long)B * S;
    t.H = H;
    return t;
}

int convert(bool store, const void* x, long long stride, const void* codes, const float* scale, int B, int S, int H, int D,
            cudaStream_t stream, bool bf16) {
    int rc = check_vectors(x, stride, codes, scale, B, S, H, D);
    if (rc != ATTN_OK || (long long)B * S * H == 0) return rc;
    const void* const all[] = {x, codes, scale};
    if (any_begins_in(all, 3)) return ATTN_ERR_INVALID_ARG;
    DeviceState dev{};
    if ((rc = device_state(&dev)) != ATTN_OK) return rc;
    const checkpoint::Tensor t = vectors_of(x, stride, codes, scale, B, S, H);
    return store ? checkpoint::launch_store(t, D, bf16, dev.num_sms, stream)
                 : checkpoint::launch_load(&t, 1, D, bf16, dev.num_sms, stream);
}

// Workspace of a backward pass from checkpoints: Q, K, V and O in 16 bits, lse, then the backward pass's own.
struct CheckpointLayout {
    size_t k = 0, v = 0, o = 0, lse = 0, bwd = 0, total = 0;
};
CheckpointLayout checkpoint_layout(int B, int Hq, int Hkv, int Sq, int Sk, int D, int mask_kind) {
    CheckpointLayout l;
    const size_t q = align_up((size_t)B * Sq * Hq * D * 2), kv = align_up((size_t)B * Sk * Hkv * D * 2);
    l.k = q;
    l.v = l.k + kv;
    l.o = l.v + kv;
    l.lse = l.o + q;
    l.bwd = l.lse + align_up((size_t)B * Hq * Sq * sizeof(float));
    l.total = l.bwd + bwd_workspace(B, Hq, Hkv, Sq, Sk, D, mask_kind);
    return l;
}

int bwd_checkpoint_impl(const void* d_o, const void* q8, const void* k8, const void* v8, const float* q_scale,
                        const float* k_scale, const float* v_scale, void* dq, void* dk, void* dv, long long dq_stride,
                        long long dk_stride, long long dv_stride, int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                        int mask_kind, const float* mask, int window, int sinks, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream, bool bf16) {
    int rc = check_sizes(B, Hq, Hkv, Sq, Sk, D);
    if (rc != ATTN_OK) return rc;
    const long long qs = (long long)Hq * D, ks = (long long)Hkv * D;
    char* const ws = static_cast<char*>(workspace);
    const bool empty = (long long)B * Sq * Hq == 0 || (long long)B * Sk == 0;
    if (empty)                                            // (no pair of a query and a key: nothing is read)
        return bwd_impl(d_o, q8, k8, v8, d_o, q_scale, dq, dk, dv, qs, ks, ks, dq_stride, dk_stride, dv_stride, B, Hq, Hkv, Sq,
                        Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes, stream, bf16);
    if ((rc = check_vectors(q8, qs, q8, q_scale, B, Sq, Hq, D)) != ATTN_OK ||
        (rc = check_vectors(k8, ks, k8, k_scale, B, Sk, Hkv, D)) != ATTN_OK ||
        (rc = check_vectors(v8, ks, v8, v_scale, B, Sk, Hkv, D)) != ATTN_OK)
        return rc;
    if (!workspace || !aligned(workspace, kWorkspaceAlign)) return ATTN_ERR_INVALID_ARG;
    if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_CAUSAL_ADDITIVE) return ATTN_ERR_INVALID_ARG;
    const CheckpointLayout l = checkpoint_layout(B, Hq, Hkv, Sq, Sk, D, mask_kind);
    if (workspace_bytes < l.total) return ATTN_ERR_INVALID_ARG;
    const void* const all[] = {dq, dk, dv, workspace, q8, k8, v8, q_scale, k_scale, v_scale, d_o, mask};
    if (any_begins_in(all, 4)) return ATTN_ERR_INVALID_ARG;
    float* const lse = reinterpret_cast<float*>(ws + l.lse);
    // Everything is checked before the first launch: the backward pass's own arguments here, the forward pass's are among them.
    rc = bwd_impl(d_o, ws, ws + l.k, ws + l.v, ws + l.o, lse, dq, dk, dv, qs, ks, ks, dq_stride, dk_stride, dv_stride, B, Hq, Hkv,
                  Sq, Sk, D, scale, mask_kind, mask, window, sinks, ws + l.bwd, l.total - l.bwd, stream, bf16, true);
    if (rc != ATTN_OK) return rc;
    DeviceState dev{};
    if ((rc = device_state(&dev)) != ATTN_OK) return rc;
    const checkpoint::Tensor t[3] = {vectors_of(ws, qs, q8, q_scale, B, Sq, Hq), vectors_of(ws + l.k, ks, k8, k_scale, B, Sk, Hkv),
                                     vectors_of(ws + l.v, ks, v8, v_scale, B, Sk, Hkv)};
    rc = checkpoint::launch_load(t, 3, D, bf16, dev.num_sms, stream);
    if (rc != ATTN_OK) return rc;
    const attn_stream_t s = reinterpret_cast<attn_stream_t>(stream);
    if (window > 0)
        rc = (bf16 ? attn_fwd_window : attn_fwd_window_f16)(ws, ws + l.k, ws + l.v, ws + l.o, lse, B, Hq, Hkv, Sq, Sk, D, scale,
                                                            window, sinks, s);
    else
        rc = (bf16 ? attn_fwd : attn_fwd_f16)(ws, ws + l.k, ws + l.v, ws + l.o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, s);
    if (rc != ATTN_OK) return rc;
    return bwd_impl(d_o, ws, ws + l.k, ws + l.v, ws + l.o, lse, dq, dk, dv, qs, ks, ks, dq_stride, dk_stride, dv_stride, B, Hq, Hkv,
                    Sq, Sk, D, scale, mask_kind, mask, window, sinks, ws + l.bwd, l.total - l.bwd, stream, bf16);
}

}  // namespace

extern "C" {

int attn_checkpoint_store(const void* x, long long x_stride, void* codes, float* scale, int B, int S, int H, int D,
                          attn_stream_t stream) {
    return convert(true, x, x_stride, codes, scale, B, S, H, D, reinterpret_cast<cudaStream_t>(stream), true);
}

int attn_checkpoint_store_f16(const void* x, long long x_stride, void* codes, float* scale, int B, int S, int H, int D,
                              attn_stream_t stream) {
    return convert(true, x, x_stride, codes, scale, B, S, H, D, reinterpret_cast<cudaStream_t>(stream), false);
}

int attn_checkpoint_load(const void* codes, const float* scale, void* x, long long x_stride, int B, int S, int H, int D,
                         attn_stream_t stream) {
    return convert(false, x, x_stride, codes, scale, B, S, H, D, reinterpret_cast<cudaStream_t>(stream), true);
}

int attn_checkpoint_load_f16(const void* codes, const float* scale, void* x, long long x_stride, int B, int S, int H, int D,
                             attn_stream_t stream) {
    return convert(false, x, x_stride, codes, scale, B, S, H, D, reinterpret_cast<cudaStream_t>(stream), false);
}

int attn_bwd_checkpoint(const void* d_o, const void* q8, const void* k8, const void* v8, const float* q_scale,
                        const float* k_scale, const float* v_scale, void* dq, void* dk, void* dv, long long dq_stride,
                        long long dk_stride, long long dv_stride, int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                        int mask_kind, const float* mask, int window, int sinks, void* workspace, size_t workspace_bytes,
                        attn_stream_t stream) {
    return bwd_checkpoint_impl(d_o, q8, k8, v8, q_scale, k_scale, v_scale, dq, dk, dv, dq_stride, dk_stride, dv_stride, B, Hq,
                               Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes,
                               reinterpret_cast<cudaStream_t>(stream), true);
}

int attn_bwd_checkpoint_f16(const void* d_o, const void* q8, const void* k8, const void* v8, const float* q_scale,
                            const float* k_scale, const float* v_scale, void* dq, void* dk, void* dv, long long dq_stride,
                            long long dk_stride, long long dv_stride, int B, int Hq, int Hkv, int Sq, int Sk, int D,
                            float scale, int mask_kind, const float* mask, int window, int sinks, void* workspace,
                            size_t workspace_bytes, attn_stream_t stream) {
    return bwd_checkpoint_impl(d_o, q8, k8, v8, q_scale, k_scale, v_scale, dq, dk, dv, dq_stride, dk_stride, dv_stride, B, Hq,
                               Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes,
                               reinterpret_cast<cudaStream_t>(stream), false);
}

size_t attn_bwd_checkpoint_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Sk, int D, int mask_kind) {
    if (check_sizes(B, Hq, Hkv, Sq, Sk, D) != ATTN_OK || mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_CAUSAL_ADDITIVE)
        return 0;
    if ((long long)B * Sq * Hq == 0 || Sk == 0) return 0;
    return checkpoint_layout(B, Hq, Hkv, Sq, Sk, D, mask_kind).total;
}

int attn_bwd(const void* d_o, const void* q, const void* k, const void* v, const void* o, const float* lse, void* dq,
             void* dk, void* dv, long long q_stride, long long k_stride, long long v_stride, long long dq_stride,
             long long dk_stride, long long dv_stride, int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
             int mask_kind, const float* mask, int window, int sinks, void* workspace, size_t workspace_bytes,
             attn_stream_t stream) {
    return bwd_impl(d_o, q, k, v, o, lse, dq, dk, dv, q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride, B, Hq,
                    Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes,
                    reinterpret_cast<cudaStream_t>(stream), true);
}

int attn_bwd_f16(const void* d_o, const void* q, const void* k, const void* v, const void* o, const float* lse, void* dq,
                 void* dk, void* dv, long long q_stride, long long k_stride, long long v_stride, long long dq_stride,
                 long long dk_stride, long long dv_stride, int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                 int mask_kind, const float* mask, int window, int sinks, void* workspace, size_t workspace_bytes,
                 attn_stream_t stream) {
    return bwd_impl(d_o, q, k, v, o, lse, dq, dk, dv, q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride, B, Hq,
                    Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes,
                    reinterpret_cast<cudaStream_t>(stream), false);
}

size_t attn_bwd_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Sk, int D, int mask_kind) {
    if (check_sizes(B, Hq, Hkv, Sq, Sk, D) != ATTN_OK || mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_CAUSAL_ADDITIVE)
        return 0;
    if ((long long)B * Sq * Hq == 0 || Sk == 0) return 0;
    return bwd_workspace(B, Hq, Hkv, Sq, Sk, D, mask_kind);
}

}  // extern "C"
