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
// are read on the device. Over short tables a CTA takes one segment whole, and the
// merge is left out (takes_whole).
//
// Memory: each warp owns a ring of stages filled by 16-byte asynchronous copies
// (16 or 32 keys and their values a stage); rows that no query sees are filled
// with zeros and tiles of such rows alone passed over, scales and all, so whatever
// stands there never enters a product. 16-byte
// chunks are XOR-swizzled by the row, which makes the ldmatrix reads of eight
// rows conflict-free.
//
// Measured (attention and merge, graph replay; the copy bandwidth of the same
// GPU is 6.70 TB/s): 16 sequences of 8192 keys, 8 K/V heads of 128, 4 query rows
// a head: e4m3 47.6 us, 5.65 TB/s, 16-bit 85.6 us, 6.28 TB/s; 32 heads of one
// row over 16-bit keys (16 x 4096, 1.07 GB) 162 us, 6.62 TB/s. What is left are
// the ends: the chain lengths - page numbers - first keys (2 us), SMs that finish
// 3 to 4 us apart, the second kernel (2). More rows over e4m3: 16 rows 53.0 us,
// 24 60.1, 32 70.3; there the tensor cores, the conversions before them and the
// softmax of a stage wait on one another.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/attn.h"
#include "attn_kernel.cuh"
#include "paged_params.h"

namespace attn {
namespace paged {

constexpr int kScanInMerge = 256;            // sequences whose units a merge CTA sums itself, one a thread
constexpr int kNoKey = 0x7fff0000;          // past every key (a sequence holds at most 2^30)
constexpr float kNoLogit = -3e38f;          // the reference before any key
constexpr float kShift = 20.f, kShiftDown = 0x1p-20f;     // 8-bit caches: see m_neg

template <int D, int CT, int NT>
struct Cfg {
    static constexpr int kElt = CT == kE4m3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElt;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kRows = 8 * NT;                         // query rows of a row block
    // Eight to twelve warps an SM hold a wide block's sums in registers; CTAs of
    // four warps cover one another's change of segment (barriers, merge, queries),
    // and stages of 32 keys (64 of 64 8-bit dims) spend one look at the queries'
    // fragments, one vote and one turn of the loop on two (four) tiles. Measured
    // over e4m3, 8 K/V heads, 16 x 8192 keys / 256 x 512 (side by side, before row
    // sums were rescaled by a root twice, which costs blocks of 20 rows and more 1%):
    //   4 rows of 128   two CTAs of eight warps, 16 keys 49.5 / 62.6 us, three of four, 32 keys 47.3 / 57.6
    //   16 rows of 128  two of eight, 16 keys 54.6 / 86.5, two of four, 32 keys 53.3 / 76.5, three of four 52.9 / 71.4
    //   20 rows of 128  one of eight, 16 keys 70.3 / 140.0, two of four 63.4 / 96.6, 32 keys 58.0 / 91.2
    //   32 rows of 128  two of four, 16 keys 77.0 / 116.5, 32 keys 69.0 / 108.5
    //   4 rows of 64    two of eight, 32 keys 29.1 / 46.6, three of four, 64 keys 28.5 / 39.3
    //   20 rows of 64   three of four, tile by tile 47.0 / 67.5, both tiles of 32 keys together 39.1 / 60.3
    // 16-bit caches, 16 x 8192: 4 rows of 64 two of eight, 16 keys 46.8, three of
    // four, 32 keys 46.1; 24 rows of 128 one of eight 92.3, two of four 94.7.
    static constexpr Plan kPlan = plan_of(D, kRows, CT);
    static constexpr int kResident = kPlan.ctas, kWarps = kPlan.warps, kKeys = kPlan.keys, kStages = kPlan.stages;
    static constexpr int kTiles = kKeys / 16;
    static constexpr int kCopies = 16 * kChunks / 32;            // 16-byte copies a lane makes for 16 keys
    static constexpr int kStageBytes = 2 * kKeys * kRowBytes;
    static constexpr int kRingBytes = kStages * kStageBytes;     // of one warp
    static constexpr bool kQShared = D * NT >= 192;              // Q fragments in shared memory, not registers
    static constexpr int kQStride = D * 2 + 16;                  // bytes of a query row: conflict-free fragment reads
    static constexpr int kScaleOff = kWarps * kRingBytes;        // [warp][stage][tile]{k, v}
    static constexpr int kKeyOff = kScaleOff + kWarps * kStages * kTiles * 8;     // [warp][stage][tile] first key
    static constexpr int kStatOff = kKeyOff + kWarps * kStages * kTiles * 4;      // [warp][row]{max, sum}
    static constexpr int kQOff = kStatOff + kWarps * kRows * 8;
    static constexpr int kFragOff = kQOff + kRows * kQStride;
    static constexpr int kShareOff = kFragOff + (kQShared ? kRows * D * 2 : 0);   // [warp]{copies', products'}
    static constexpr int kIssueOff = kShareOff + kWarps * 2 * 80;    // [warp] what a stage's copies need of a share
    static constexpr int kRowOff = kIssueOff + kWarps * 32;  // [row] score factor; [row]{factor, place in O} of the merge
    static constexpr int kSmemBytes = kRowOff + kRows * 16;
    static constexpr int kMergeTiles = kStageBytes / (8 * D * 4);    // n-tiles that a stage of the ring takes at once
    static_assert(kMergeTiles >= 1, "a warp's rows are merged through one stage of its ring");
    static_assert(kUnit % kKeys == 0, "a stage lies inside one unit");
    static_assert(kQOff % 16 == 0 && kFragOff % 16 == 0, "16-byte accesses");
    static_assert(kResident * (kSmemBytes + 1024 + 128) <= 233472, "shared memory budget");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2(const void* at) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(at) : "memory");
}
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

// Two 16x16 matrices of bytes, transposed: lanes 0..15 and 16..31 give the rows
// of each. Lane 4g + t receives bytes 4t..4t+3 of column g in r[0] (second
// matrix: r[2]) and of column g + 8 in r[1] (r[3]).
__device__ __forceinline__ void ldmatrix_bytes_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
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

// The key of a 16-key tile that stands in row m of the products. An 8-bit tile's
// values come from ldmatrix with four consecutive keys a lane, which are the
// products' columns 2t, 2t + 1, 2t + 8 and 2t + 9: so those rows hold the keys
// 4t..4t+3.
template <bool E4M3>
__device__ __forceinline__ int key_of_row(int m) {
    return E4M3 ? ((m & 6) << 1) + (m & 1) + ((m >> 2) & 2) : m;
}

// Byte offset of 16-byte chunk c of row r in a swizzled stage. The eight rows
// that one step of an ldmatrix reads lie in different banks: rows 0..7 or 8..15,
// and for an 8-bit tile's keys also those of key_of_row, {0, 1, 4, 5, 8, ...}
// and {2, 3, 6, 7, 10, ...}.
template <int ROWB, bool E4M3>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    if (ROWB == 64) {                                            // two rows share a 128-byte line
        const int line = r >> 1, x = ((line >> 1) & 1) | (((line ^ (line >> 2)) & 1) << 1);
        return (uint32_t)(line * 128 + (((((r & 1) << 2) + c) ^ x) << 4));
    }
    const int x = E4M3 ? (r & 1) | ((r >> 1) & 2) | (((r << 1) ^ (r >> 1)) & 4) : r & 7;
    return (uint32_t)(r * ROWB + ((c ^ x) << 4));
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

// The schedule. Every non-empty segment counts its units and, where the CTAs
// have several units each, kLead more for what a CTA pays to begin a segment
// (its queries, the merge of the one before); each CTA takes an equal range of
// the positions of all segments, end to end. With few
// units there is no lead and no more CTAs than units. Either way every CTA
// between a segment's first and last one holds a part of it.
constexpr int kLead = 4;
__device__ __forceinline__ int lead_of(const AttendParams& p, int units) { return units >= 8 * p.ctas ? kLead : 0; }
__device__ __forceinline__ int span_of(int units, int lead) { return units > 0 ? units + lead : 0; }
__device__ __forceinline__ int working_ctas(const AttendParams& p, int total) { return min(p.ctas, total); }
// (32-bit divisions: they stand on the path to the first copy.)
struct Ranges {
    int each, more;      // positions of a CTA; the first `more` CTAs have one more
    __device__ __forceinline__ Ranges(int total, int ctas) : each(total / ctas), more(total - each * ctas) {}
    __device__ __forceinline__ int start(int cta) const { return cta * each + min(cta, more); }
    // The CTA whose range holds position x.
    __device__ __forceinline__ int owner(int x) const {
        const int big = more * (each + 1);
        return x < big ? x / (each + 1) : more + (x - big) / each;
    }
};

// One segment's share of a CTA: units [u0, u1) of the key list of row block rb
// of K/V head hk of sequence b.
struct Share {
    int b, base;         // the sequence and the first unit of its segments
    KeyList list;
    int hk, rb, u0, u1;
    int next;            // position after the share
    int pos_lo, pos_hi;  // positions of the row block's first and last query
    int kv_end;          // keys at or past it are hidden from every row
    int w_lo;            // keys before it are hidden too, but for the sinks
};

static_assert(sizeof(Share) <= 80, "the size the shared-memory layout gives it");

// The first share with a unit in positions [x, x_end), searching onwards from
// s.b (whose list is s.list); false if there is none.
template <int ROWS>
__device__ __forceinline__ bool locate(const AttendParams& p, int segs, int lead, int x, int x_end, Share& s) {
    bool bad;
    int seg;
    for (;;) {
        if (x >= x_end) return false;
        const int span = span_of(s.list.units, lead);
        if (x >= s.base + span * segs) {                          // the sequence is done, or empty
            s.base += span * segs;
            if (++s.b >= p.B) return false;                       // (only if the lengths changed under the call)
            s.list = key_list(p, s.b, bad);
            continue;
        }
        seg = (x - s.base) / span;
        const int off = x - s.base - seg * span;
        s.u0 = max(0, off - lead);
        s.u1 = min(s.list.units, off + x_end - x - lead);
        s.next = min(x_end, s.base + (seg + 1) * span);
        if (s.u1 > s.u0) break;
        x = s.next;
    }
    s.hk = p.row_blocks == 1 ? seg : seg / p.row_blocks;
    s.rb = seg - s.hk * p.row_blocks;
    const int r0 = s.rb * ROWS;
    const int i0 = r0 == 0 ? 0 : r0 / p.group, i1 = min(p.Sq == 1 ? 0 : min(p.rows - 1, r0 + ROWS - 1) / p.group, s.list.ql - 1);
    s.pos_lo = s.list.kv - s.list.ql + i0;
    s.pos_hi = s.list.kv - s.list.ql + i1;
    s.kv_end = i0 < s.list.ql ? max(0, s.pos_hi + 1) : 0;
    s.w_lo = p.window > 0 ? s.pos_lo - p.window + 1 : 0;
    return true;
}

// Rows of a segment without any key: o = 0, lse = -inf.
template <int D, int ROWS, int THREADS>
__device__ __forceinline__ void fill_rows(const AttendParams& p, int b, int seg, int ql, int tid) {
    const int hk = seg / p.row_blocks, r0 = (seg - hk * p.row_blocks) * ROWS;
    for (int w = tid; w < ROWS * (D / 8); w += THREADS) {
        const int row = r0 + w / (D / 8), c = w % (D / 8), i = row / p.group;
        if (row >= p.rows || i >= ql) continue;
        const int h = hk * p.group + (row - i * p.group);
        reinterpret_cast<uint4*>(p.o)[(((size_t)b * p.Sq + i) * p.Hq + h) * (D / 8) + c] = make_uint4(0u, 0u, 0u, 0u);
        if (c == 0) p.lse[((size_t)b * p.Hq + h) * p.Sq + i] = -INFINITY;
    }
}

template <int D, int CT, int NT>
__global__ void __launch_bounds__(Cfg<D, CT, NT>::kWarps * 32, Cfg<D, CT, NT>::kResident)
    paged_attend_kernel(const AttendParams p) {
    using C = Cfg<D, CT, NT>;
    constexpr int kThreads = C::kWarps * 32;
    constexpr int kSteps = D / 16;                                // products of 16 dims
    constexpr bool kBf = CT == kBf16;                             // operand type of the products
    extern __shared__ __align__(1024) uint8_t smem_raw[];          // the XOR of chunk offsets needs 256-byte stages
    __shared__ int2 s_scan[C::kWarps];
    __shared__ Share s_begin;                                     // (b, base, list) where the CTA's range begins
    __shared__ int s_range[2];                                    // the schedule's lead, the range's end
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    wait_for_inputs();
    let_next_start();
    uint8_t* const ring = smem_raw + warp * C::kRingBytes;
    const uint32_t ring_a = ptx::smem_addr(ring);
    float* const scales = reinterpret_cast<float*>(smem_raw + C::kScaleOff) + warp * C::kStages * C::kTiles * 2;
    volatile int* const keys_sh = reinterpret_cast<int*>(smem_raw + C::kKeyOff) + warp * C::kStages * C::kTiles;
    float2* const stats = reinterpret_cast<float2*>(smem_raw + C::kStatOff);
    uint8_t* const q_sh = smem_raw + C::kQOff;
    uint2* const frag_sh = reinterpret_cast<uint2*>(smem_raw + C::kFragOff);
    float* const row_sh = reinterpret_cast<float*>(smem_raw + C::kRowOff);
    float2* const total_sh = reinterpret_cast<float2*>(smem_raw + C::kRowOff) + C::kRows;

    // The page numbers come into L2 while the lengths are on their way (a line a
    // thread; a table past that is fetched as it is needed).
    {
        const long long line = (long long)blockIdx.x * kThreads + tid;
        if (line * 32 < (long long)p.B * p.max_pages) prefetch_l2(p.block_table + line * 32);
    }
    // ---- where this CTA's range begins: a scan over the sequences' units
    const int segs = p.Hkv * p.row_blocks;                        // segments of a sequence
    int x, x_end;
    if (p.whole) {
        const int b = blockIdx.x / segs, seg = blockIdx.x - b * segs;
        bool bad;
        const KeyList list = key_list(p, b, bad);
        if (bad && seg == 0 && tid == 0) atomicOr(p.status, kStatusBadIndex);
        if (list.units == 0) {
            fill_rows<D, C::kRows, kThreads>(p, b, seg, list.ql, tid);
            return;
        }
        x = seg * list.units;
        x_end = x + list.units;
        if (tid == 0) {
            s_begin.b = b;
            s_begin.base = 0;
            s_begin.list = list;
            s_range[0] = 0;
            s_range[1] = x_end;
        }
    } else {
        const int per = (p.B + kThreads - 1) / kThreads;
        const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
        KeyList list{};
        int mine = 0, mine_n = 0;                                     // units, and sequences with any
        for (int b = b_lo; b < b_hi; ++b) {
            bool bad;
            list = key_list(p, b, bad);
            mine += list.units;
            mine_n += list.units > 0;
            if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
        }
        int incl = mine, incl_n = mine_n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o), n = __shfl_up_sync(0xffffffffu, incl_n, o);
            if (lane >= o) incl += v, incl_n += n;
        }
        if (lane == 31) s_scan[warp] = make_int2(incl, incl_n);
        __syncthreads();
        int before = incl - mine, before_n = incl_n - mine_n, total = 0, total_n = 0;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            const int2 v = s_scan[w];
            if (w < warp) before += v.x, before_n += v.y;
            total += v.x, total_n += v.y;
        }
        const int lead = lead_of(p, total * segs);
        before = (before + before_n * lead) * segs;
        mine = (mine + mine_n * lead) * segs;
        total = (total + total_n * lead) * segs;
        const int ctas = working_ctas(p, total);
        const Ranges ranges(total, max(ctas, 1));
        const bool works = (int)blockIdx.x < ctas;
        x = works ? ranges.start(blockIdx.x) : total;
        x_end = works ? ranges.start(blockIdx.x + 1) : total;
        if (tid == 0) {
            s_range[0] = lead;
            s_range[1] = x_end;
        }
        const bool note = blockIdx.x == 0 && p.B > kScanInMerge;      // the merge reads the offsets of a large batch
        if (note || (before <= x && x < before + mine)) {
            int at = before;
            for (int b = b_lo; b < b_hi; ++b) {
                bool bad;
                if (per > 1) list = key_list(p, b, bad);
                const int n = span_of(list.units, lead) * segs;
                if (note) p.base[b] = at;
                if (at <= x && x < at + n) {
                    s_begin.b = b;
                    s_begin.base = at;
                    s_begin.list = list;
                }
                at += n;
            }
            if (note && b_hi == p.B && b_lo < b_hi) {
                p.base[p.B] = at;
                p.base[p.B + 1] = lead;
            }
        }
    }
    __syncthreads();
    if (x >= x_end) return;

    // Where a lane's pieces lie in a swizzled stage. Copy c of a 16-key tile is
    // chunk lane % kChunks of row c * (32 / kChunks) + lane / kChunks; the
    // swizzle repeats every 8 rows (16 rows of 8-bit values), so a few offsets
    // describe all copies. The ldmatrix rows likewise: chunk 2c is the XOR of
    // c << 5 with chunk 0.
    constexpr int kCopyRows = 32 / C::kChunks;                     // rows of one copy
    constexpr int kPeriod = CT == kE4m3 ? 16 : 8;
    constexpr int kCopyKinds = kPeriod / kCopyRows;
    uint32_t copy_off[kCopyKinds];
#pragma unroll
    for (int c = 0; c < kCopyKinds; ++c)
        copy_off[c] = swizzled<C::kRowBytes, CT == kE4m3>(c * kCopyRows + lane / C::kChunks, lane % C::kChunks);
    auto copy_to = [&](int c) {
        return copy_off[c % kCopyKinds] + (uint32_t)(c / kCopyKinds * kCopyKinds * kCopyRows * C::kRowBytes);
    };
    const uint32_t k_off = swizzled<C::kRowBytes, CT == kE4m3>(key_of_row<CT == kE4m3>(lane & 15), lane >> 4);
    const uint32_t v_off = CT == kE4m3
                               ? swizzled<C::kRowBytes, true>(lane & 15, lane >> 4)
                               : swizzled<C::kRowBytes, false>((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
    const int sinks = p.window > 0 ? p.sinks : 0;

    // ---- the copies run ahead of the products, across segments: `ld` is the
    // share they are in, ld_i its next stage. A segment then begins with its
    // first stages already on their way, and the memory stays busy while the
    // last segment's rows are merged.
    // Both shares stand in shared memory, one copy a warp: they would take some
    // 25 registers.
    Share& ld = reinterpret_cast<Share*>(smem_raw + C::kShareOff)[2 * warp];
    Share& cur = reinterpret_cast<Share*>(smem_raw + C::kShareOff)[2 * warp + 1];
    if (lane == 0) ld = s_begin;
    __syncwarp();
    int ld_x = x, ld_i = 0, ld_n = 0, ld_stage = 0;
    bool ld_more = false;
    const uint32_t page_bytes = ((uint32_t)p.Hkv << p.page_shift) * C::kRowBytes;
    uint32_t head_off = 0;                                        // of the share's head in a page, and the lane's chunk
    // What a stage's copies need of the share, as two vectors beside it: keys
    // {count, offset of the gap, first before it, first past it (less the
    // offset)}, {end, start of the window, sequence, head}.
    int4* const ld_v = reinterpret_cast<int4*>(smem_raw + C::kIssueOff) + 2 * warp;
    // Page numbers (-1: no key that a query of the block sees, or out of range)
    // and scales of the next 32 / kTiles stages, one 16-key tile a lane. A unit at
    // either end of the window may hold tiles that nobody sees: neither their page
    // numbers nor their scales are looked at (a scale multiplies weights of zero
    // too, and a page behind the window may have left the table).
    constexpr int kBatch = 32 / C::kTiles;
    int ids = -1;
    float2 sc = make_float2(0.f, 0.f);
    int sc_slot = -1, sc_lane = 0;                                // the stage whose scales are still to be put down
    auto stages_of = [](int units) { return (units * kUnit + C::kWarps * C::kKeys - 1) / (C::kWarps * C::kKeys); };
    auto enter = [&]() {                                          // the share at ld_x
        Share s = ld;
        ld_more = locate<C::kRows>(p, segs, s_range[0], ld_x, s_range[1], s);
        if (!ld_more) return;
        __syncwarp();
        if (lane == 0) {
            ld = s;
            const int gap = max(0, (s.list.sink_units - s.u0) * kUnit);
            ld_v[0] = make_int4((s.u1 - s.u0) * kUnit, gap, s.u0 * kUnit,
                                (s.u0 - s.list.sink_units + s.list.first) * kUnit);
            ld_v[1] = make_int4(s.kv_end, s.w_lo, s.b, s.hk);
        }
        __syncwarp();
        ld_i = 0;
        ld_n = stages_of(s.u1 - s.u0);
        head_off = ((uint32_t)s.hk << p.page_shift) * C::kRowBytes + lane * 16;
        // The queries are read when the products get there; by then they are in L2.
        if (warp == 0) {
            const int r0 = s.rb * C::kRows, row = r0 + lane;
            const int i = row / p.group;
            if (lane < C::kRows && row < p.rows && i < s.list.ql) {
                const uint16_t* q = p.q + ((long long)s.b * p.Sq + i) * p.q_stride +
                                    (long long)(s.hk * p.group + (row - i * p.group)) * D;
                const int pos = min(max(s.list.kv - s.list.ql + i, 0), p.max_pos - 1);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) prefetch_l2(q + 64 * c);
                if (p.rope && row == max(r0, i * p.group)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) prefetch_l2(p.rope + (size_t)pos * D + 32 * c);
                }
            }
        }
    };
    enter();
    if (!ld_more) return;                                         // nothing but leads in its range
    auto issue = [&]() {
        if (CT == kE4m3 && sc_slot >= 0) {
            // (a stage late, when they have arrived; the products come later still)
            if ((lane ^ sc_lane) < C::kTiles) reinterpret_cast<float2*>(scales)[sc_slot + (lane ^ sc_lane)] = sc;
            sc_slot = -1;
        }
        if (ld_more) {
            const int4 u = ld_v[0], w = ld_v[1];
            if (ld_i % kBatch == 0) {
                const int off = ((ld_i + lane / C::kTiles) * C::kWarps + warp) * C::kKeys + lane % C::kTiles * 16;
                const int key = off + (off < u.y ? u.z : u.w);
                ids = -1;
                sc = make_float2(1.f, 1.f);
                if (off < u.x && key < w.x && (key + 16 > w.y || key < sinks)) {
                    ids = p.block_table[(size_t)w.z * p.max_pages + (key >> p.page_shift)];
                    if ((unsigned)ids >= (unsigned)p.n_pages) {
                        atomicOr(p.status, kStatusBadIndex);
                        ids = -1;
                    } else if (CT == kE4m3) {
                        const uint64_t at = (uint64_t)(uint32_t)ids * (uint32_t)p.Hkv + w.w;
                        sc = make_float2(__ldcg(p.k_scale + at), __ldcg(p.v_scale + at));
                    }
                }
            }
            const int off0 = (ld_i * C::kWarps + warp) * C::kKeys, first = ld_i % kBatch * C::kTiles;
            const uint32_t dst = ring_a + ld_stage * C::kStageBytes;
#pragma unroll
            for (int m = 0; m < C::kTiles; ++m) {
                const int id = __shfl_sync(0xffffffffu, ids, first + m);
                const int k0 = off0 + 16 * m + (off0 + 16 * m < u.y ? u.z : u.w);
                if (lane == 0) keys_sh[ld_stage * C::kTiles + m] = id >= 0 ? k0 : kNoKey;
                if (C::kTiles == 1 && id < 0) continue;       // (its stage is passed over)
                const uint32_t slot = (uint32_t)(k0 & ((1 << p.page_shift) - 1));
                const uint64_t at = (uint64_t)(uint32_t)max(id, 0) * page_bytes + (head_off + slot * C::kRowBytes);
                const uint8_t* ks = static_cast<const uint8_t*>(p.k_cache) + at;
                const uint8_t* vs = static_cast<const uint8_t*>(p.v_cache) + at;
                const uint32_t kd = dst + m * 16 * C::kRowBytes, vd = kd + C::kKeys * C::kRowBytes;
                if ((C::kTiles == 1 || id >= 0) && k0 + 16 <= w.x && (k0 >= w.y || k0 + 16 <= sinks)) {
#pragma unroll
                    for (int c = 0; c < C::kCopies; ++c) {
                        cp_async16(kd + copy_to(c), ks + c * 512);
                        cp_async16(vd + copy_to(c), vs + c * 512);
                    }
                } else {
                    // rows that no query of the block sees are filled with zeros
#pragma unroll
                    for (int c = 0; c < C::kCopies; ++c) {
                        const int key = k0 + (c * 32 + lane) / C::kChunks;
                        const bool take = id >= 0 && key < w.x && (key >= w.y || key < sinks);
                        cp_async16(kd + copy_to(c), ks + c * 512, take);
                        cp_async16(vd + copy_to(c), vs + c * 512, take);
                    }
                }
            }
            sc_slot = ld_stage * C::kTiles;
            sc_lane = first;
            if (++ld_i == ld_n) {
                ld_x = ld.next;
                enter();
            }
        }
        cp_async_commit();
        ld_stage = ld_stage + 1 == C::kStages ? 0 : ld_stage + 1;
    };
    if (lane == 0) cur = ld;
    __syncwarp();

    // ---- queries: fetched (a 16-byte piece and its angles, kQItems a thread)
    // before the previous rows are merged, then rotated, rounded to their 16-bit
    // type and put into shared memory.
    constexpr int kQItems = (C::kRows * (D / 8) + kThreads - 1) / kThreads;
    const bool bf = CT == kE4m3 ? p.q_bf16 : kBf;
    uint4 q_raw[kQItems];
    float4 q_turn[kQItems][2];
    auto fetch_q = [&](const Share& s) {
#pragma unroll
        for (int j = 0; j < kQItems; ++j) {
            const int w = tid + j * kThreads, r = w / (D / 8), d = (w - r * (D / 8)) * 8;
            const int row = s.rb * C::kRows + r, i = row / p.group;
            q_raw[j] = make_uint4(0u, 0u, 0u, 0u);
            q_turn[j][0] = q_turn[j][1] = make_float4(1.f, 0.f, 1.f, 0.f);
            if (r < C::kRows && row < p.rows && i < s.list.ql) {
                q_raw[j] = *reinterpret_cast<const uint4*>(p.q + ((long long)s.b * p.Sq + i) * p.q_stride +
                                                           (long long)(s.hk * p.group + (row - i * p.group)) * D + d);
                if (p.rope) {
                    int pos = s.list.kv - s.list.ql + i;
                    if (pos >= p.max_pos) {
                        if (d == 0) atomicOr(p.status, kStatusBadIndex);
                        pos = p.max_pos - 1;
                    }
                    const float4* at = reinterpret_cast<const float4*>(p.rope) + (size_t)max(pos, 0) * (D / 4) + d / 4;
                    q_turn[j][0] = __ldg(at);
                    q_turn[j][1] = __ldg(at + 1);
                }
            }
        }
    };
    auto store_q = [&]() {
#pragma unroll
        for (int j = 0; j < kQItems; ++j) {
            const int w = tid + j * kThreads, r = w / (D / 8), d = (w - r * (D / 8)) * 8;
            uint32_t v[4] = {q_raw[j].x, q_raw[j].y, q_raw[j].z, q_raw[j].w};
            if (p.rope) {
                const float4 a = q_turn[j][0], c = q_turn[j][1];
                v[0] = bf ? rotate_pair<true>(v[0], a.x, a.y) : rotate_pair<false>(v[0], a.x, a.y);
                v[1] = bf ? rotate_pair<true>(v[1], a.z, a.w) : rotate_pair<false>(v[1], a.z, a.w);
                v[2] = bf ? rotate_pair<true>(v[2], c.x, c.y) : rotate_pair<false>(v[2], c.x, c.y);
                v[3] = bf ? rotate_pair<true>(v[3], c.z, c.w) : rotate_pair<false>(v[3], c.z, c.w);
            }
            if (r < C::kRows)
                *reinterpret_cast<uint4*>(q_sh + r * C::kQStride + d * 2) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    };
    fetch_q(cur);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) issue();

    uint32_t qf[C::kQShared ? 1 : kSteps][C::kQShared ? 1 : NT][2];
    int st = 0;                                                   // stage of the next products
    for (;;) {
        const int r0 = cur.rb * C::kRows, pos0 = cur.list.kv - cur.list.ql;
        const int pos_lo = cur.pos_lo, pos_hi = cur.pos_hi;
        store_q();
        __syncthreads();
        // B fragments. With an 8-bit cache the queries become f16 values, each
        // row scaled by a power of two to lie in [-2, 2]: exact down to 2^-24 of
        // the row's largest value, whatever the row's magnitude. Where the
        // fragments stand in shared memory each n-tile is one warp's work.
        float cf[NT][2];                                          // log2 units per raw score, rows 2t and 2t + 1
        auto fragments = [&](int n, uint32_t (&w)[kSteps][2]) -> float {
            const uint8_t* src = q_sh + (8 * n + g) * C::kQStride;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                // the dims that the keys' fragments of the step hold
                if (CT == kE4m3) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src + (16 * s + 4 * t) * 2);
                    w[s][0] = v.x;
                    w[s][1] = v.y;
                } else {
                    w[s][0] = *reinterpret_cast<const uint32_t*>(src + (16 * s + 2 * t) * 2);
                    w[s][1] = *reinterpret_cast<const uint32_t*>(src + (16 * s + 8 + 2 * t) * 2);
                }
            }
            if (CT != kE4m3) return 1.f;
            float top = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 a = widen16(w[s][h], bf);
                    top = fmaxf(top, fmaxf(fabsf(a.x), fabsf(a.y)));
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -120), 120);
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 a = widen16(w[s][h], bf);
                    w[s][h] = ptx::pack_f16x2(a.x * f, a.y * f);
                }
            return __uint_as_float((uint32_t)(127 + e) << 23);    // of row g
        };
        if constexpr (C::kQShared) {
            if (warp < NT) {
                uint32_t w[kSteps][2];
                const float back = fragments(warp, w);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) frag_sh[(s * NT + warp) * 32 + lane] = make_uint2(w[s][0], w[s][1]);
                if (t == 0) row_sh[8 * warp + g] = p.scale_log2 * back;
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                cf[n][0] = row_sh[8 * n + 2 * t];
                cf[n][1] = row_sh[8 * n + 2 * t + 1];
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t w[kSteps][2];
                const float back = fragments(n, w);
                cf[n][0] = p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t);
                cf[n][1] = p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    qf[s][n][0] = w[s][0];
                    qf[s][n][1] = w[s][1];
                }
            }
        }

        float acc[kSteps][NT][4];                                 // O^T
        // Rows 2t, 2t + 1 of each n-tile: minus the reference in use (log2 units)
        // and this lane's part of the sum of 2^(logit - reference). Over an 8-bit
        // cache the reference follows logit + log2(value scale), so that what goes
        // to the tensor cores, weight * scale, is largest where it matters most,
        // whatever the scales of other pages. The weights alone then reach
        // 2^(8 + kShift) / scale: FP32 holds them and their sum for scales from
        // 2^-72 to 2^120 (values under smaller scales, below 2^-63, fade to zero),
        // and where it is brought to a higher reference the factor, down to 2^-220,
        // is applied as its root twice; alone it would leave FP32's range.
        // Below any logit at first, so that no weight needs a special case.
        float m_neg[NT][2], l_sum[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m_neg[n][0] = m_neg[n][1] = -kNoLogit;
            l_sum[n][0] = l_sum[n][1] = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) acc[s][n][0] = acc[s][n][1] = acc[s][n][2] = acc[s][n][3] = 0.f;
        }

        const int n_it = stages_of(cur.u1 - cur.u0);
        for (int i = 0; i < n_it; ++i) {
            cp_async_wait<C::kStages - 2>();
            __syncwarp();
            issue();
            if (C::kStages == 2) __syncwarp();                // (it puts down this stage's scales)
            // All tiles of a stage together: one look at the queries' fragments, one
            // vote. The first key of each; kNoKey: nothing there, or a page out of
            // range (its rows are zeros, and hidden).
            constexpr int M = C::kTiles;
            int k0[M];
            bool none = true, whole = true;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                k0[m] = keys_sh[st * M + m];
                none &= k0[m] == kNoKey;
                whole &= k0[m] + 15 <= pos_lo && (k0[m] >= pos_hi - p.window + 1 || p.window == 0 || k0[m] + 16 <= sinks);
            }
            if (!none) {
                const uint32_t ka = ring_a + st * C::kStageBytes + k_off;
                const uint32_t va = ring_a + st * C::kStageBytes + C::kKeys * C::kRowBytes + v_off;
                // ---- S^T = K Q^T
                float s[M][NT][4];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[m][n][0] = s[m][n][1] = s[m][n][2] = s[m][n][3] = 0.f;
#pragma unroll
                for (int c = 0; c < C::kChunks / 2; ++c) {
                    uint32_t r[M][4];
#pragma unroll
                    for (int m = 0; m < M; ++m) ldmatrix4<false>(r[m], (ka ^ (uint32_t)(c << 5)) + m * 16 * C::kRowBytes);
                    if (CT == kE4m3) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t a[M][4];
#pragma unroll
                            for (int m = 0; m < M; ++m) {
                                a[m][0] = e4m3_lo(r[m][2 * h]);
                                a[m][1] = e4m3_lo(r[m][2 * h + 1]);
                                a[m][2] = e4m3_hi(r[m][2 * h]);
                                a[m][3] = e4m3_hi(r[m][2 * h + 1]);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint2 q2;
                                if constexpr (C::kQShared)
                                    q2 = frag_sh[((2 * c + h) * NT + n) * 32 + lane];
                                else
                                    q2 = make_uint2(qf[2 * c + h][n][0], qf[2 * c + h][n][1]);
#pragma unroll
                                for (int m = 0; m < M; ++m)
                                    mma16816<false>(s[m][n], a[m][0], a[m][1], a[m][2], a[m][3], q2.x, q2.y);
                            }
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint2 q2;
                            if constexpr (C::kQShared)
                                q2 = frag_sh[(c * NT + n) * 32 + lane];
                            else
                                q2 = make_uint2(qf[c][n][0], qf[c][n][1]);
#pragma unroll
                            for (int m = 0; m < M; ++m)
                                mma16816<kBf>(s[m][n], r[m][0], r[m][1], r[m][2], r[m][3], q2.x, q2.y);
                        }
                    }
                }
                // ---- logits in log2 units; hidden keys to -inf
                float vs[M], lv[M], f[M][NT][2];                   // f: log2 units per value of s
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    float ks = 1.f;
                    vs[m] = 1.f;
                    lv[m] = 0.f;
                    if (CT == kE4m3) {
                        const float2 kv2 = *reinterpret_cast<const float2*>(scales + (st * M + m) * 2);
                        ks = kv2.x;
                        vs[m] = kv2.y * kShiftDown;
                        lv[m] = fminf(fmaxf(__log2f(fabsf(kv2.y)), -72.f), 120.f) - kShift;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) f[m][n][e] = CT == kE4m3 ? cf[n][e] * ks : p.scale_log2;
                }
                if (!whole) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int pos = pos0 + (r0 + 8 * n + 2 * t + e) / p.group;
                            const int lo = p.window > 0 ? pos - p.window : -1;
#pragma unroll
                            for (int m = 0; m < M; ++m) {
                                const int j0 = k0[m] + key_of_row<CT == kE4m3>(g), j1 = j0 + (CT == kE4m3 ? 2 : 8);
                                const bool h0 = j0 > pos || (j0 <= lo && j0 >= sinks), h1 = j1 > pos || (j1 <= lo && j1 >= sinks);
                                s[m][n][e] = h0 ? -INFINITY : s[m][n][e] * f[m][n][e];
                                s[m][n][2 + e] = h1 ? -INFINITY : s[m][n][2 + e] * f[m][n][e];
                                f[m][n][e] = 1.f;
                            }
                        }
                }
                // The reference may trail the true maximum by 2^8 (the weights
                // then reach 2^8, far inside 16-bit range), so most stages need
                // one vote instead of the reduction and the rescaling.
                bool grow = false;
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            grow |= fmaf(fmaxf(s[m][n][e], s[m][n][2 + e]), f[m][n][e], m_neg[n][e]) > kRescaleThreshold - lv[m];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(s[0][n][e], s[0][n][2 + e]) * f[0][n][e] + lv[0];
#pragma unroll
                            for (int m = 1; m < M; ++m)
                                mx = fmaxf(mx, fmaxf(s[m][n][e], s[m][n][2 + e]) * f[m][n][e] + lv[m]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                            mx = fmaxf(mx, -m_neg[n][e]);
                            // (the root of the factor, twice: see m_neg)
                            const float root = ptx::ex2(0.5f * (-m_neg[n][e] - mx)), alpha = root * root;
                            m_neg[n][e] = -mx;
                            l_sum[n][e] = l_sum[n][e] * root * root;
#pragma unroll
                            for (int d = 0; d < kSteps; ++d) {
                                acc[d][n][e] *= alpha;
                                acc[d][n][2 + e] *= alpha;
                            }
                        }
                    }
                }
                // ---- weights; P in f16 (bf16 for a bf16 cache), summed before that rounding
                uint32_t pb[M][NT][2];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float w[4];
                        float(&x)[4] = s[m][n];
                        ptx::fma2(w[0], w[1], x[0], x[1], f[m][n][0], f[m][n][1], m_neg[n][0], m_neg[n][1]);
                        ptx::fma2(w[2], w[3], x[2], x[3], f[m][n][0], f[m][n][1], m_neg[n][0], m_neg[n][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = ptx::ex2(w[e]);
                        ptx::add2(l_sum[n][0], l_sum[n][1], l_sum[n][0], l_sum[n][1], w[0], w[1]);
                        ptx::add2(l_sum[n][0], l_sum[n][1], l_sum[n][0], l_sum[n][1], w[2], w[3]);
                        if (CT == kE4m3) {
                            ptx::mul2(w[0], w[1], w[0], w[1], vs[m], vs[m]);
                            ptx::mul2(w[2], w[3], w[2], w[3], vs[m], vs[m]);
                        }
                        pb[m][n][0] = transpose8x8(kBf ? ptx::pack_bf16x2(w[0], w[1]) : ptx::pack_f16x2(w[0], w[1]));
                        pb[m][n][1] = transpose8x8(kBf ? ptx::pack_bf16x2(w[2], w[3]) : ptx::pack_f16x2(w[2], w[3]));
                    }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int c = 0; c < C::kChunks / 2; ++c) {
                        const uint32_t at = (va ^ (uint32_t)(c << 5)) + m * 16 * C::kRowBytes;
                        uint32_t r[4];
                        if (CT == kE4m3) {
                            ldmatrix_bytes_trans(r, at);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t a0 = e4m3_lo(r[2 * h]), a1 = e4m3_lo(r[2 * h + 1]),
                                               a2 = e4m3_hi(r[2 * h]), a3 = e4m3_hi(r[2 * h + 1]);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma16816<false>(acc[2 * c + h][n], a0, a1, a2, a3, pb[m][n][0], pb[m][n][1]);
                            }
                        } else {
                            ldmatrix4<true>(r, at);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma16816<kBf>(acc[c][n], r[0], r[1], r[2], r[3], pb[m][n][0], pb[m][n][1]);
                        }
                    }
            }
            st = st + 1 == C::kStages ? 0 : st + 1;
        }

        // ---- the next share's queries set out
        Share now = cur;
        Share s = now;
        const bool more = locate<C::kRows>(p, segs, s_range[0], now.next, s_range[1], s);
        if (more) {
            __syncwarp();
            if (lane == 0) cur = s;
            __syncwarp();
            if (NT == 1) fetch_q(s);
        }
        // ---- merge the warps through the stage that was read last (the others
        // hold the next segment's keys): first the maxima and sums, so that each
        // warp can write its O^T in the units of the common maximum, then O^T,
        // kMergeTiles n-tiles at a time.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_sum[n][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (g == 0) stats[warp * C::kRows + 8 * n + 2 * t + e] = make_float2(-m_neg[n][e], l);
            }
        __syncthreads();
        const bool full = now.u0 == 0 && now.u1 == now.list.units;
        float* slot = p.part + (size_t)(2 * blockIdx.x + (now.u0 == 0 ? 1 : 0)) * C::kRows * (D + 2);
        float to_common = 0.f;                                    // of row `lane`
        if (lane < C::kRows) {
            float mx = kNoLogit;
#pragma unroll
            for (int v = 0; v < C::kWarps; ++v) mx = fmaxf(mx, stats[v * C::kRows + lane].x);
            to_common = ptx::ex2(stats[warp * C::kRows + lane].x - mx + (CT == kE4m3 ? kShift : 0.f));
            if (warp == 0) {
                // The row's factor and place in the output (-1: none); its sum.
                float sum = 0.f, inv = 1.f;
#pragma unroll
                for (int v = 0; v < C::kWarps; ++v) {
                    const float2 s2 = stats[v * C::kRows + lane];
                    const float root = ptx::ex2(0.5f * (s2.x - mx));
                    sum = fmaf(s2.y * root, root, sum);
                }
                const int row = r0 + lane, i = row / p.group;
                const bool live = row < p.rows && i < now.list.ql;
                const int h = now.hk * p.group + (row - i * p.group);
                if (!full) {
                    slot[C::kRows * D + lane] = mx;
                    slot[C::kRows * (D + 1) + lane] = sum;
                } else if (live) {
                    inv = sum != 0.f ? 1.f / sum : 0.f;               // 0: no key was visible
                    p.lse[((size_t)now.b * p.Hq + h) * p.Sq + i] =
                        sum != 0.f ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
                }
                total_sh[lane] = make_float2(inv, __int_as_float(live ? i * p.Hq + h : -1));
            }
        }
        const int m_stage = st == 0 ? C::kStages - 1 : st - 1;
        float* const mine_o = reinterpret_cast<float*>(ring + m_stage * C::kStageBytes);
        uint16_t* const out = p.o + (size_t)now.b * p.Sq * p.Hq * D;
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += C::kMergeTiles) {
#pragma unroll
            for (int n = n0; n < NT && n < n0 + C::kMergeTiles; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = __shfl_sync(0xffffffffu, to_common, 8 * n + 2 * t + e);
                    float* const row = mine_o + (8 * (n - n0) + 2 * t + e) * D;
#pragma unroll
                    for (int d = 0; d < kSteps; ++d) {
                        row[(16 * d + g) ^ (t << 3)] = acc[d][n][e] * f;     // XOR: spreads the rows over the banks
                        row[(16 * d + 8 + g) ^ (t << 3)] = acc[d][n][2 + e] * f;
                    }
                }
            }
            __syncthreads();
            constexpr int kItems = D / 4;                         // float4 of a row
            const int rows = 8 * min(C::kMergeTiles, NT - n0);
            for (int w = tid; w < rows * kItems; w += kThreads) {
                const int c = w / kItems, d = (w - c * kItems) * 4, col = 8 * n0 + c;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int v = 0; v < C::kWarps; ++v) {
                    const float4 a = *reinterpret_cast<const float4*>(
                        reinterpret_cast<const float*>(smem_raw + v * C::kRingBytes + m_stage * C::kStageBytes) + c * D +
                        (d ^ (((c & 7) >> 1) << 3)));
                    o.x += a.x;
                    o.y += a.y;
                    o.z += a.z;
                    o.w += a.w;
                }
                if (full) {
                    const float2 ri = total_sh[col];
                    const int at = __float_as_int(ri.y);
                    if (at >= 0) {
                        uint2 r;
                        r.x = bf ? ptx::pack_bf16x2(o.x * ri.x, o.y * ri.x) : ptx::pack_f16x2(o.x * ri.x, o.y * ri.x);
                        r.y = bf ? ptx::pack_bf16x2(o.z * ri.x, o.w * ri.x) : ptx::pack_f16x2(o.z * ri.x, o.w * ri.x);
                        *reinterpret_cast<uint2*>(out + (size_t)at * D + d) = r;
                    }
                } else {
                    *reinterpret_cast<float4*>(slot + col * D + d) = o;
                }
            }
            // The stage is free for the next tiles; after the last ones, for the
            // copies, which come after the barrier below.
            if (n0 + C::kMergeTiles < NT) __syncthreads();
        }
        if (!more) break;
        if (NT > 1) fetch_q(s);                                   // (earlier it would cost registers the sums need)
    }
    cp_async_wait<0>();
}

// Merges the parts of the segments that several CTAs share, and fills the rows
// of sequences without a key:
//   m = max_c m_c,  l = sum_c l_c 2^(m_c - m),  o = sum_c o_c 2^(m_c - m) / l.
// One warp per row; a lane holds D / 32 dims. Bound by latency: a segment has a
// few parts, all of whose loads are in flight at once; some 2 us behind the
// attention, of which the launch, the schedule and the lengths run beside it.
template <int D, int RB>
__global__ void __launch_bounds__(256) paged_merge_kernel(const AttendParams p, bool bf16) {
    constexpr int kPer = D / 32;
    __shared__ int2 s_scan[8], s_mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int segs = p.Hkv * p.row_blocks;
    const int b = blockIdx.x / segs, seg = blockIdx.x - b * segs;
    int total, first, units, lead;
    if (p.B <= kScanInMerge) {
        // The sequences' units, one a thread: lengths are the step's inputs, so
        // this needs nothing of the attention kernel and runs beside it.
        bool bad;
        const int mine = (int)threadIdx.x < p.B ? key_list(p, threadIdx.x, bad).units : 0;
        int incl = mine, incl_n = mine > 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o), n = __shfl_up_sync(0xffffffffu, incl_n, o);
            if (lane >= o) incl += v, incl_n += n;
        }
        if (lane == 31) s_scan[warp] = make_int2(incl, incl_n);
        __syncthreads();
        int before = incl - mine, before_n = incl_n - (mine > 0), total_n = 0;
        total = 0;
        for (int w = 0; w < 8; ++w) {
            const int2 v = s_scan[w];
            if (w < warp) before += v.x, before_n += v.y;
            total += v.x, total_n += v.y;
        }
        lead = lead_of(p, total * segs);
        if ((int)threadIdx.x == b) s_mine = make_int2(before + before_n * lead, mine);
        __syncthreads();
        total = (total + total_n * lead) * segs;
        first = s_mine.x * segs;
        units = s_mine.y;
        wait_for_inputs();
    } else {
        wait_for_inputs();
        total = p.base[p.B];
        lead = p.base[p.B + 1];
        first = p.base[b];
        const int span = (p.base[b + 1] - first) / segs;
        units = span > 0 ? span - lead : 0;
    }
    let_next_start();
    int c0 = 0, c1 = 0;
    if (units > 0) {
        const int span = units + lead;
        const Ranges ranges(total, working_ctas(p, total));
        c0 = ranges.owner(first + seg * span + lead);
        c1 = min(ranges.owner(first + (seg + 1) * span - 1), p.ctas - 1);     // (as above)
        if (c0 == c1) return;
    }
    const int hk = seg / p.row_blocks, rb = seg - hk * p.row_blocks;
    int ql = p.q_lens ? p.q_lens[b] : p.Sq;
    ql = min(max(ql, 0), p.Sq);
    for (int col = warp; col < RB; col += 8) {
        const int row = rb * RB + col, i = row / p.group;
        if (row >= p.rows || i >= ql) continue;
        const int h = hk * p.group + (row - i * p.group);
        float mx = kNoLogit, sum = 0.f, o[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = 0.f;
        if (units > 0) {
            // Eight parts at a time, their loads all in flight before any is used.
            constexpr size_t kStride = (size_t)RB * (D + 2);
            for (int c = c0; c <= c1; c += 8) {
                float pm[8], pl[8], po[8][kPer];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    pm[j] = kNoLogit;
                    pl[j] = 0.f;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) po[j][e] = 0.f;
                    if (c + j <= c1) {
                        const float* slot = p.part + (size_t)(2 * (c + j) + (c + j == c0 ? 1 : 0)) * kStride;
                        pm[j] = slot[RB * D + col];
                        pl[j] = slot[RB * (D + 1) + col];
#pragma unroll
                        for (int e = 0; e < kPer; ++e) po[j][e] = slot[col * D + lane * kPer + e];
                    }
                }
                float m8 = mx;
#pragma unroll
                for (int j = 0; j < 8; ++j) m8 = fmaxf(m8, pm[j]);
                const float r0 = ptx::ex2(0.5f * (mx - m8)), f0 = r0 * r0;      // (see m_neg)
                mx = m8;
                sum = sum * r0 * r0;
#pragma unroll
                for (int e = 0; e < kPer; ++e) o[e] *= f0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float r = ptx::ex2(0.5f * (pm[j] - mx)), f = r * r;
                    sum = fmaf(pl[j] * r, r, sum);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) o[e] = fmaf(po[j][e], f, o[e]);
                }
            }
        }
        const float inv = sum != 0.f ? 1.f / sum : 0.f;         // 0: no key was visible
        uint16_t* dst = p.o + (((size_t)b * p.Sq + i) * p.Hq + h) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = bf16 ? ptx::pack_bf16x2(o[e] * inv, o[e + 1] * inv)
                                                         : ptx::pack_f16x2(o[e] * inv, o[e + 1] * inv);
        if (lane == 0)
            p.lse[((size_t)b * p.Hq + h) * p.Sq + i] = sum != 0.f ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
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
    const bool bf16 = CT == kBf16 || (CT == kE4m3 && p.q_bf16);
    if (launch_early(kernel, p.ctas, C::kWarps * 32, C::kSmemBytes, stream, p) != cudaSuccess) return ATTN_ERR_CUDA;
    if (!p.whole &&
        launch_early(paged_merge_kernel<D, C::kRows>, (unsigned)(p.B * p.Hkv * p.row_blocks), 256, 0, stream, p, bf16) !=
            cudaSuccess)
        return ATTN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int CT>
int launch_attend(bool (&attr_set)[2][4], const AttendParams& p, int D, cudaStream_t stream) {
    bool(&set)[4] = attr_set[D == 128];
    switch (block_rows(p.rows)) {
        case 8:
            return D == 128 ? launch_instance<128, CT, 1>(set[0], p, stream) : launch_instance<64, CT, 1>(set[0], p, stream);
        case 16:
            return D == 128 ? launch_instance<128, CT, 2>(set[1], p, stream) : launch_instance<64, CT, 2>(set[1], p, stream);
        case 24:
            return D == 128 ? launch_instance<128, CT, 3>(set[2], p, stream) : launch_instance<64, CT, 3>(set[2], p, stream);
        default:
            return D == 128 ? launch_instance<128, CT, 4>(set[3], p, stream) : launch_instance<64, CT, 4>(set[3], p, stream);
    }
}

}  // namespace paged
}  // namespace attn
