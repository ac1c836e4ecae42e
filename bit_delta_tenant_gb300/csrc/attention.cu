// attention.cu -- attention of one new token per sequence over a paged
// key-value cache, split over the cache's length and joined.
//
//   o = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),  s_j = scale * q . K_j
//
// Bound: HBM (each K and V element is used by the few query heads that share
// its KV head).  One pass over the cache with a running maximum and sum.
//
// Work.  The keys of every (sequence, KV head) are cut into blocks of a tile per warp
// (64 keys in bf16, 128 in 8 bits); the blocks of the whole batch, numbered sequence by
// sequence, head by head, are split evenly over the resident CTAs, so ragged lengths
// leave no CTA idle and the host needs no length.  A CTA streams its range; where the
// range ends inside a (sequence, head) it leaves the unnormalised output, maximum and sum
// of its part in the workspace; the last of eight neighbouring parts to arrive joins
// them in key order, the last of eight such joins those, and so on.  No CTA waits for
// another.  Where no sequence can be long, each warp takes whole heads and nothing is joined.
//
// A warp.  Each of the four warps owns a tile of a block's keys and keeps its own
// running state; 16 keys of one page and head are one contiguous piece of
// memory, copied with cp.async into the warp's own ring (swizzled so that the
// fragment loads meet no bank conflict), the page ids read a batch ahead.
// S = Q K^T has the query heads as rows; O^T += V^T P^T has them as columns, so
// S's accumulator is P^T's operand as it stands and 8 heads fill a column tile.
// mma.sync, not tcgen05: 4 to 16 rows of a 128-row tile would be used, and at HBM's rate
// the products take a sixth of mma.sync's (bf16, at most 8 heads to a KV head: 32 products
// for 8 KB of K and V, 14 us of the 88 below).
//
// Rounding.  P enters as a 16-bit part and its 16-bit remainder: bf16 (2^-16 of a
// weight) beside a bf16 V, fp16 (2^-21, or 2^-40 of the largest) beside an e4m3 V,
// which fp16 holds exactly.  An e4m3 V's scale is folded into the
// weight before the maximum is taken, so that no weight exceeds 2^15; its K is
// multiplied as it stands, by q in two e4m3 parts: q is scaled by a power of two
// so that its row's largest value lies in [128, 256), where the parts hold a bf16
// value's 8 bits exactly (values far below the largest to 2^-21 of it); with at most 8
// heads the second part takes rows 8..15 of the same product.  Accumulation is
// fp32 in every product (measured for the e4m3 one: 2^-25 of sum |q k|).
//
// Measured (head_dim 128): 130001 tokens, 64 and 8 heads, bf16 89 us (6.0 TB/s: SMs' streams end between 64 and
// 82 us, then the joins), 8 bits 56 (4.8 TB/s); sequences of up to 8191 tokens, lengths spread in their logarithm, 32
// and 8 heads, 8 bits: 64 of them 34 us (3.6 TB/s), 200 86 (4.4 TB/s), one to six heads to a CTA that drains its ring
// at each head's end before the next head's first copy; 200 of them in bf16 122 (6.1 TB/s); 777 tokens, bf16 8.2 us,
// a chain of latencies.  More than 16 query heads to a KV head read it once per 16: 64 sequences of up to 4000 tokens,
// one KV head, bf16, 16 query heads 13.1 us, 48 17.2.
#include <cuda_fp8.h>

#include <algorithm>

#include "bd_device.cuh"
#include "bd_internal.h"

namespace bd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;  // query heads of one tile
constexpr int kMaxCtasPerSm = 3;
constexpr int kDepth = 2;  // tiles in a warp's ring: one in use, one in flight
constexpr int64_t kMaxKeys = 1 << 30;  // the division by the page size is exact, positions stay int32
constexpr int kSlotFloats = kRows * 128 + 2 * kRows;  // a part's output, maxima and sums
constexpr int64_t kAloneKeys = 512;  // keys of a head that a warp may be given by itself
constexpr int kSetup = 2;  // what a (sequence, head) costs a CTA beside its blocks, in blocks
constexpr int kFan = 8;      // parts joined at a time
constexpr int kLevels = 4;   // enough for kFan^4 parts
constexpr uint32_t kNoPage = 0xFFFFFFFFu;

struct AttnArgs {
    const uint8_t *q, *ck, *cv, *ck_scale, *cv_scale;
    const int32_t *page_table, *lengths;
    uint8_t *out;
    float *lse, *parts;
    int32_t *counters;  // [kLevels][level_counters], one per slot
    unsigned *status;
    int64_t n_pages;
    int32_t n_seqs, max_pages, kv_heads, page_size, q_heads, group, subs, window;
    int32_t level_counters;
    uint32_t page_tiles, page_magic;  // page_size / 16, and ceil(2^32 / that) for divisions by it
    float scale_log2;                 // scale * log2(e): scores are kept in base 2
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool full) {
    const int n = full ? 16 : 0;  // 0: nothing is read, 16 zero bytes are written
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 bytes as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t four, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float ex2(float x) {  // 2^x, 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A bf16 pair times `up` as e4m3 bytes, and 16 times what they leave as e4m3 bytes.  In fp16 the
// scaled values (at most 256, 8 bits) and the differences are exact down to 2^-24.
__device__ __forceinline__ void split_e4m3(uint32_t pair, float up, uint32_t &hi, uint32_t &lo) {
    const __half2 x = __floats2half2_rn(bf16lo_to_f32(pair) * up, bf16hi_to_f32(pair) * up);
    const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const __half2 left = __hmul2(__hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3))), __float2half2_rn(16.f));
    hi = h;
    lo = __nv_cvt_halfraw2_to_fp8x2(left, __NV_SATFINITE, __NV_E4M3);
}

// Byte offset of 16-byte chunk c of row r in a tile of kRow-byte rows: eight rows of one
// chunk column fall into eight different 16-byte bank groups.
template <int kRow>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    if constexpr (kRow == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) * 16);
    return r * kRow + ((c ^ (r & 7)) * 16);
}

// What a sequence's query sees: keys [start, len), cut into `blocks` blocks from block `first`; with
// a head's setup and join that is `units` of work per head.
struct Span {
    int32_t start, len, first, blocks, units;
};
template <int kBlock>
__device__ __forceinline__ Span span_of(const AttnArgs &a, int64_t b) {
    const int64_t most = min(static_cast<int64_t>(a.max_pages) * a.page_size, kMaxKeys);
    int64_t len = a.lengths[b];
    if (len < 0 || len > most) {
        flag_status(a.status, kDevBadIndex);
        len = len < 0 ? 0 : most;
    }
    Span s;
    s.len = static_cast<int32_t>(len);
    s.start = a.window > 0 && len > a.window ? s.len - a.window : 0;
    s.first = s.start / kBlock;
    s.blocks = (s.len + kBlock - 1) / kBlock - s.first;
    s.units = s.blocks > 0 ? s.blocks + kSetup : 0;
    return s;
}

// x / y of whole numbers; the quick form where both fit 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    if ((x | y) >> 32) return x / y;
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
}

// `total` units over at most `most` CTAs, the first `extra` of them with one unit more.
struct Share {
    int64_t ctas, each, extra;
    __device__ __forceinline__ Share(int64_t total, int64_t most) {
        ctas = min(most, total);
        each = ctas ? quotient(total, ctas) : 0;
        extra = total - each * ctas;
    }
    __device__ __forceinline__ int64_t begin(int64_t c) const { return each * c + min(c, extra); }
    __device__ __forceinline__ int64_t owner(int64_t unit) const {  // the CTA whose range holds the unit
        const int64_t head = (each + 1) * extra;
        return unit < head ? quotient(unit, each + 1) : extra + quotient(unit - head, each);
    }
};

__device__ __forceinline__ int64_t warp_scan(int64_t v) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (static_cast<int>(threadIdx.x % 32) >= o) v += u;
    }
    return v;
}

// Weights are kept times 2^kLift: beside an e4m3 V they are fp16, whose range below 1 ends at 2^-24, and a token whose V
// has a small scale weighs little beside one with a large scale, yet is all there is in columns where that one is 0.
template <bool kE4m3>
constexpr float kLift = kE4m3 ? 15.f : 0.f;  // the largest is 2^15

template <bool kE4m3>
constexpr int kTileOf = kE4m3 ? 32 : 16;  // keys of a warp's step: 8 KB of K and V at head_dim 128 in either type
template <bool kE4m3>
constexpr int kBlockOf = kWarps *kTileOf<kE4m3>;  // keys of a work item
template <int kDim, bool kE4m3>
constexpr int stage_bytes() {  // K tile, V tile, and their scale bytes
    return 2 * kTileOf<kE4m3> * kDim * (kE4m3 ? 1 : 2) + (kE4m3 ? 2 * kTileOf<kE4m3> : 0);
}
template <int kDim, bool kE4m3>
constexpr int smem_bytes() {
    return kWarps * kDepth * stage_bytes<kDim, kE4m3>();
}

// CTAs per SM: the second column tile of more than 8 heads takes the registers of the third CTA.
template <bool kPack>
constexpr int kCtasOf = kPack ? 3 : 2;

// The heads of units begin .. end, or alone: of heads begin, begin + every warp of the grid, .. below end by this warp.
// kPack: at most 8 query heads.
template <int kDim, bool kE4m3, bool kPack, bool alone>
__device__ __forceinline__ void stream(const AttnArgs &a, uint8_t *smem, const Share &share, int64_t begin, int64_t end, int64_t b,
                                       int64_t units_before) {
    constexpr int kTile = kTileOf<kE4m3>, kBlock = kBlockOf<kE4m3>;
    constexpr int kSub = kTile / 16;              // 16-key pieces of a tile, each within one page
    constexpr int kRow = kDim * (kE4m3 ? 1 : 2);  // bytes of one key
    constexpr int kChunks = kRow / 16;
    constexpr int kPiece = 16 * kRow;             // bytes of 16 keys
    constexpr int kTileBytes = kSub * kPiece;
    constexpr int kStage = stage_bytes<kDim, kE4m3>();
    constexpr int kHalves = kPack ? 1 : 2;   // column tiles of 8 heads
    constexpr int kSteps = kRow / 32;        // k steps of Q K^T: 32 bytes of a key each
    constexpr int kRowTiles = kDim / 16;     // row tiles of V^T P^T
    constexpr int kBatch = 32 / kSub;        // tiles whose page ids a warp holds at a time
    constexpr int stride_keys = alone ? kTile : kBlock;  // from a warp's tile to its next
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ float s_jm[kFan][kRows], s_jl[kFan][kRows];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t4 = lane % 4;
    const int vheads = a.kv_heads * a.subs;
    Span sp = span_of<kBlock>(a, b);
    int vh = alone ? 0 : static_cast<int>(quotient(begin - units_before * vheads, sp.units));
    const uint32_t ring = smem_u32(smem) + warp * (kDepth * kStage);
    // Lane offsets that repeat: the swizzle turns with the row, so a copy has kTurns of them and a
    // fragment load one per chunk pair within 128 bytes; everything else is a constant.
    constexpr int kTurns = kChunks / 4, kPairs = kSteps < 4 ? kSteps : 4;
    uint32_t copy_at[kTurns], load_at[kPairs];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) copy_at[i] = ring + tile_at<kRow>((lane + 32 * i) / kChunks, lane % kChunks);
#pragma unroll
    for (int k = 0; k < kPairs; ++k)
        load_at[k] = ring + tile_at<kRow>(lane % 8 + lane / 16 * 8, 2 * k + lane / 8 % 2);
    const uint8_t *ring_ptr = smem + warp * (kDepth * kStage);

    for (int64_t at = begin; at < end;) {
        if (alone) {
            b = quotient(at, vheads);
            vh = static_cast<int>(at - b * vheads);
            sp = span_of<kBlock>(a, b);
        }
        // this head's units start at i0, its setup first; what lies in this CTA's range of its blocks
        const int64_t i0 = units_before * vheads + static_cast<int64_t>(vh) * sp.units;
        const int64_t stop = alone ? at + static_cast<int64_t>(gridDim.x) * kWarps : min(end, i0 + sp.units);
        const int blk = alone ? 0 : max(0, static_cast<int>(at - i0) - kSetup);
        const int n = alone ? (sp.len + kTile - 1) / kTile - sp.start / kTile : max(0, static_cast<int>(stop - i0) - kSetup) - blk;
        if (n > 0) {
        const int kvh = vh / a.subs, row0 = vh % a.subs * kRows;
        const int rows = min(kRows, a.group - row0);
        const int64_t head0 = b * a.q_heads + kvh * a.group + row0;
        const int key_first = alone ? sp.start / kTile * kTile : (sp.first + blk) * kBlock + warp * kTile;  // tile j: + j * stride_keys

        // 16-key piece `lane` of the batch of tiles from j0: its page id
        const int32_t *table = a.page_table + b * a.max_pages;
        auto piece_of = [&](int j0) { return static_cast<uint32_t>(key_first + (j0 + lane / kSub) * stride_keys) / 16 + lane % kSub; };
        auto page_index = [&](uint32_t piece) { return a.page_tiles == 1 ? piece : __umulhi(piece, a.page_magic); };
        auto fetch_page = [&](int j0) {
            const uint32_t p = piece_of(j0);
            const bool on = j0 + lane / kSub < n && static_cast<int>(p * 16) < sp.len && static_cast<int>(p * 16 + 16) > sp.start;
            const bool there = on && in_bounds(b < a.n_seqs && page_index(p) < static_cast<uint32_t>(a.max_pages), a.status);
            return there ? table[page_index(p)] : 0;
        };
        // its place in the pool, in units of 16 keys
        auto place_of = [&](int j0, int32_t page) {
            if (page < 0 || page >= a.n_pages) {
                flag_status(a.status, kDevBadIndex);
                return kNoPage;
            }
            const uint32_t p = piece_of(j0);
            return (static_cast<uint32_t>(page) * a.kv_heads + kvh) * a.page_tiles + (p - page_index(p) * a.page_tiles);
        };
        int32_t next_pages = fetch_page(0);

        // Q fragments: rows are heads, and with kPack rows 8..15 the second part of e4m3 queries
        constexpr int kParts = kE4m3 && !kPack ? 2 : 1;
        uint32_t qa[kParts][kSteps][kPack && !kE4m3 ? 2 : 4];
        float rscale[2] = {a.scale_log2, a.scale_log2};
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
            const bool on = g + half * 8 < rows &&
                            in_bounds(head0 + g + half * 8 < static_cast<int64_t>(a.n_seqs) * a.q_heads, a.status);
            const uint8_t *src = a.q + (head0 + g + half * 8) * (kDim * 2);
            if constexpr (!kE4m3) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t v = on ? *reinterpret_cast<const uint32_t *>(src + k * 32 + i * 16 + t4 * 4) : 0;
                        qa[0][k][kPack ? i : 2 * i + half] = v;
                    }
            } else {
                uint32_t v[kSteps][2][2], top2 = 0;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {  // columns 32 k + 16 i + 4 t .. + 3
                        const uint2 x = on ? *reinterpret_cast<const uint2 *>(src + k * 64 + i * 32 + t4 * 8) : make_uint2(0, 0);
                        v[k][i][0] = x.x, v[k][i][1] = x.y;
                        // magnitudes of bf16 pairs compare as whole numbers, NaN above infinity
                        top2 = __vmaxu2(top2, __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu));
                    }
                top2 = __vmaxu2(top2, __shfl_xor_sync(0xFFFFFFFFu, top2, 1));
                top2 = __vmaxu2(top2, __shfl_xor_sync(0xFFFFFFFFu, top2, 2));
                const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
                // 2^(e - 127) <= largest < 2^(e - 126); rows of zeros, next to zero or next to infinity take e = 127
                int e = static_cast<int>(top >> 7);
                e = e < 27 || e > 227 ? 127 : e;
                const float up = __uint_as_float(static_cast<uint32_t>(254 + 7 - e) << 23);  // to [128, 256)
                // neither infinity nor NaN has an e4m3 form that keeps it through a product: such a head is NaN throughout
                rscale[half] = top >= 0x7F80u ? NAN : a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 7) << 23);
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t hi[2], lo[2];
#pragma unroll
                        for (int w = 0; w < 2; ++w) split_e4m3(v[k][i][w], up, hi[w], lo[w]);
                        if constexpr (kPack) {
                            qa[0][k][2 * i] = hi[0] | hi[1] << 16, qa[0][k][2 * i + 1] = lo[0] | lo[1] << 16;
                        } else {
                            qa[0][k][2 * i + half] = hi[0] | hi[1] << 16, qa[1][k][2 * i + half] = lo[0] | lo[1] << 16;
                        }
                    }
            }
        }

        float o[kRowTiles][kHalves][4] = {};
        float m[kHalves], l[kHalves];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) m[h] = -INFINITY, l[h] = 0.f;

        uint32_t places = place_of(0, next_pages);
        next_pages = fetch_page(kBatch);
        uint32_t bad = 0;  // pieces in the ring whose page id is out of range
        auto load = [&](int j, const int slot) {
            if (j >= n) return;
            if (j > 0 && j % kBatch == 0) {
                places = place_of(j, next_pages);
                next_pages = fetch_page(j + kBatch);
            }
            const int key0 = key_first + j * stride_keys;
            if (key0 >= sp.len || key0 + kTile <= sp.start) return;
            const uint32_t to = slot * kStage;
            const bool inside = key0 >= sp.start && key0 + kTile <= sp.len;
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                uint32_t place = __shfl_sync(0xFFFFFFFFu, places, j % kBatch * kSub + u);
                const bool good = place != kNoPage &&
                                  in_bounds(place < static_cast<uint64_t>(a.n_pages) * a.kv_heads * a.page_tiles, a.status);
                if (!good) bad |= 1u << (slot * kSub + u), place = 0;
                const uint8_t *ks = a.ck + static_cast<int64_t>(place) * kPiece + lane * 16;
                const uint8_t *vs = a.cv + static_cast<int64_t>(place) * kPiece + lane * 16;
                // chunk lane + 32 i of the piece; the offsets repeat after kTurns copies of 512 bytes
                if (inside && good) {
#pragma unroll
                    for (int i = 0; i < 16 * kChunks / 32; ++i) {
                        const uint32_t d = copy_at[i % kTurns] + to + u * kPiece + i / kTurns * (kTurns * 512);
                        cp_async16(d, ks + i * 512);
                        cp_async16(d + kTileBytes, vs + i * 512);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16 * kChunks / 32; ++i) {
                        const uint32_t d = copy_at[i % kTurns] + to + u * kPiece + i / kTurns * (kTurns * 512);
                        const int key = key0 + u * 16 + (lane + 32 * i) / kChunks;
                        const bool seen = good && key < sp.len && key >= sp.start;
                        cp_async16(d, ks + i * 512, seen);
                        cp_async16(d + kTileBytes, vs + i * 512, seen);
                    }
                }
                if constexpr (kE4m3)
                    if (lane < 2)
                        cp_async16(ring + to + 2 * kTileBytes + lane * kTile + u * 16,
                                   (lane ? a.cv_scale : a.ck_scale) + static_cast<int64_t>(place) * 16, good);
            }
        };
        // one tile: the copy of the next one is started, then this one is waited for and used
        auto step = [&](int j, const int slot) {
            load(j + 1, slot ^ 1);
            cp_commit();
            cp_wait<1>();
            __syncwarp();
            const int key0 = key_first + j * stride_keys;
            if (key0 < sp.len && key0 + kTile > sp.start) {
                const uint32_t to = slot * kStage;
                const uint8_t *vp = ring_ptr + to + kTileBytes;
                [[maybe_unused]] const uint8_t *scales = vp + kTileBytes;
                // 8 keys x 16 bytes per matrix: a chunk pair for keys 0..7, then for keys 8..15 of a piece
                auto pair_at = [&](int u, int k) { return load_at[k % kPairs] + to + u * kPiece + k / kPairs * 128; };
                float s[2 * kSub][4] = {};
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        uint32_t r[4];
                        ldsm4(r, pair_at(u, k));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float(&d)[4] = s[2 * u + i];
                            if constexpr (kE4m3)
                                mma_e4m3(d, qa[0][k][0], qa[0][k][1], qa[0][k][2], qa[0][k][3], r[2 * i], r[2 * i + 1]);
                            else if constexpr (kPack)
                                mma16<false>(d, qa[0][k][0], 0, qa[0][k][1], 0, r[2 * i], r[2 * i + 1]);
                            else
                                mma16<false>(d, qa[0][k][0], qa[0][k][1], qa[0][k][2], qa[0][k][3], r[2 * i], r[2 * i + 1]);
                        }
                    }
                if constexpr (kE4m3 && !kPack) {  // the second parts of q, 1/16 of the weight
                    float s2[2 * kSub][4] = {};
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
#pragma unroll
                        for (int u = 0; u < kSub; ++u) {
                            uint32_t r[4];
                            ldsm4(r, pair_at(u, k));
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                mma_e4m3(s2[2 * u + i], qa[1][k][0], qa[1][k][1], qa[1][k][2], qa[1][k][3], r[2 * i],
                                         r[2 * i + 1]);
                        }
#pragma unroll
                    for (int i = 0; i < 2 * kSub; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[i][c] = fmaf(s2[i][c], 0.0625f, s[i][c]);
                }
                // scores in base 2; V's scale, as a factor and as its exponent
                float vscale[2 * kSub][2], vexp[2 * kSub][2];
#pragma unroll
                for (int i = 0; i < 2 * kSub; ++i) {
                    float ks[2] = {1.f, 1.f};
                    if constexpr (kE4m3) {
                        const uint32_t kb = *reinterpret_cast<const uint16_t *>(scales + i * 8 + t4 * 2);
                        const uint32_t vb = *reinterpret_cast<const uint16_t *>(scales + kTile + i * 8 + t4 * 2);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            ks[c] = __uint_as_float((kb >> 8 * c & 0xFFu) << 23);
                            vscale[i][c] = __uint_as_float((vb >> 8 * c & 0xFFu) << 23);
                            // a byte below the smallest scale's, as in slots never written: no weight overflows
                            vexp[i][c] = fmaxf(__uint_as_float(0x4B000000u | (vb >> 8 * c & 0xFFu)) - (8388608.f + 127.f), -60.f);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if constexpr (kE4m3 && kPack) s[i][c] = fmaf(s[i][2 + c], 0.0625f, s[i][c]);
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            s[i][2 * h + c] *= kE4m3 ? ks[c] * rscale[h] : rscale[h];
                    }
                }
                const uint32_t bad_here = bad >> slot * kSub & ((1u << kSub) - 1);
                if (key0 < sp.start || key0 + kTile > sp.len || bad_here) {
#pragma unroll
                    for (int i = 0; i < 2 * kSub; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int key = key0 + i * 8 + t4 * 2 + c;
                            const bool seen = key < sp.len && key >= sp.start && !(bad_here >> i / 2 & 1);
#pragma unroll
                            for (int h = 0; h < kHalves; ++h) s[i][2 * h + c] = seen ? s[i][2 * h + c] : -INFINITY;
                            if (kE4m3 && !seen) vscale[i][c] = vexp[i][c] = 0.f;  // the byte may be anything
                        }
                }
                float fix[kHalves];
                bool moved = false;
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    float top = m[h];
#pragma unroll
                    for (int i = 0; i < 2 * kSub; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            top = fmaxf(top, kE4m3 ? s[i][2 * h + c] + vexp[i][c] : s[i][2 * h + c]);
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const float now = top == -INFINITY ? 0.f : top, base = now - kLift<kE4m3>;  // nothing yet: all weights 0
                    fix[h] = ex2(m[h] - now);
                    moved |= fix[h] != 1.f;
                    m[h] = top;
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 2 * kSub; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float e = ex2(s[i][2 * h + c] - base);
                            sum += e;
                            s[i][2 * h + c] = kE4m3 ? e * vscale[i][c] : e;
                        }
                    l[h] = fmaf(l[h], fix[h], sum);
                }
                if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {  // columns 2t, 2t+1 of O^T: the factors sit in those heads' lanes
                        const float f0 = __shfl_sync(0xFFFFFFFFu, fix[h], t4 * 8);
                        const float f1 = __shfl_sync(0xFFFFFFFFu, fix[h], t4 * 8 + 4);
#pragma unroll
                        for (int c = 0; c < kRowTiles; ++c) {
                            o[c][h][0] *= f0, o[c][h][1] *= f1;
                            o[c][h][2] *= f0, o[c][h][3] *= f1;
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    uint32_t p[kHalves][2], p2[kHalves][2];  // P^T and its remainder
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float x = s[2 * u + i][2 * h], y = s[2 * u + i][2 * h + 1];
                            if constexpr (kE4m3) {
                                p[h][i] = pack_half2(x, y);
                                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p[h][i]));
                                p2[h][i] = pack_half2(x - f.x, y - f.y);
                            } else {
                                p[h][i] = pack_bf16x2(x, y);
                                p2[h][i] = pack_bf16x2(x - bf16lo_to_f32(p[h][i]), y - bf16hi_to_f32(p[h][i]));
                            }
                        }
                    if constexpr (kE4m3) {
                        // rows 2t, 2t+1, 2t+8, 2t+9; the lane's piece of a row holds columns g * kDim / 8 ..,
                        // rows g and g + 8 of row tile c are its columns 2c and 2c + 1
                        constexpr int kWords = kDim / 32;
                        uint32_t w[4][kWords];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = u * 16 + t4 * 2 + i % 2 + i / 2 * 8;
                            if constexpr (kWords == 4) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(vp + tile_at<kRow>(r, g));
                                w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
                            } else {
                                const uint2 x = *reinterpret_cast<const uint2 *>(vp + tile_at<kRow>(r, g / 2) + g % 2 * 8);
                                w[i][0] = x.x, w[i][1] = x.y;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kWords; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t v[4];  // two columns' bytes of two keys, side by side
                                e4m3x4_to_half2x2(__byte_perm(w[0][i], w[1][i], e ? 0x7362 : 0x5140), v[0], v[1]);
                                e4m3x4_to_half2x2(__byte_perm(w[2][i], w[3][i], e ? 0x7362 : 0x5140), v[2], v[3]);
#pragma unroll
                                for (int h = 0; h < kHalves; ++h) {
                                    mma16<true>(o[2 * i + e][h], v[0], v[1], v[2], v[3], p[h][0], p[h][1]);
                                    mma16<true>(o[2 * i + e][h], v[0], v[1], v[2], v[3], p2[h][0], p2[h][1]);
                                }
                            }
                    } else {
#pragma unroll
                        for (int c = 0; c < kRowTiles; ++c) {
                            uint32_t v[4];
                            ldsm4_trans(v, pair_at(u, c) + kTileBytes);
#pragma unroll
                            for (int h = 0; h < kHalves; ++h) {
                                mma16<false>(o[c][h], v[0], v[1], v[2], v[3], p[h][0], p[h][1]);
                                mma16<false>(o[c][h], v[0], v[1], v[2], v[3], p2[h][0], p2[h][1]);
                            }
                        }
                    }
                }
            }
            bad &= ~(((1u << kSub) - 1) << slot * kSub);
            __syncwarp();  // the slot may be refilled
        };
        load(0, 0);
        cp_commit();
        for (int j = 0; j < n; j += 2) {
            step(j, 0);
            if (j + 1 < n) step(j + 1, 1);
        }
        cp_wait<0>();
        __syncwarp();
        if (!alone) __syncthreads();

        // the warps' states in shared memory, [warp][row][kStride], where a warp alone keeps to its ring
        constexpr int kUsed = 8 * kHalves;
        constexpr int kStride = kDim + 4;  // rows of heads 2t fall into different banks
        static_assert(kUsed * kStride * 4 <= kDepth * kStage && kStage % 16 == 0);
        float *merge = reinterpret_cast<float *>(smem);
        float *own = alone ? reinterpret_cast<float *>(smem + warp * (kDepth * kStage)) : merge + warp * kUsed * kStride;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
            if (t4 == 0) s_m[warp][g + 8 * h] = m[h], s_l[warp][g + 8 * h] = l[h];
            float *mine = own + (8 * h + 2 * t4) * kStride;
#pragma unroll
            for (int e = 0; e < 2; ++e, mine += kStride) {
                if constexpr (kE4m3) {
#pragma unroll
                    for (int c = 0; c < kRowTiles; c += 2)
                        *reinterpret_cast<float4 *>(mine + g * (kDim / 8) + 2 * c) =
                            make_float4(o[c][h][e], o[c][h][2 + e], o[c + 1][h][e], o[c + 1][h][2 + e]);
                } else {
#pragma unroll
                    for (int c = 0; c < kRowTiles; ++c) mine[c * 16 + g] = o[c][h][e], mine[c * 16 + g + 8] = o[c][h][2 + e];
                }
            }
        }
        auto finish = [&](int r, int d, float4 x, float top, float sum) {  // four columns of a row, and once its lse
            if (!in_bounds(head0 + r < static_cast<int64_t>(a.n_seqs) * a.q_heads, a.status)) return;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2 *>(a.out + ((head0 + r) * kDim + d) * 2) =
                make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
            if (a.lse && d == 0) a.lse[head0 + r] = (top - kLift<kE4m3> + log2f(sum)) * 0.693147180559945f;
        };
        if (alone) {
            __syncwarp();
            for (int i = lane; i < rows * (kDim / 4); i += 32) {
                const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
                finish(r, d, *reinterpret_cast<const float4 *>(own + r * kStride + d), s_m[warp][r], s_l[warp][r]);
            }
            __syncwarp();  // the ring is free again
            at = stop;
            continue;
        }
        __syncthreads();
        const bool whole = blk == 0 && n == sp.blocks;
        [[maybe_unused]] auto in_slots = [&](const float *slot) {  // one whole slot of the workspace
            const int64_t at = slot - a.parts;
            return in_bounds(at >= 0 && at <= (a.level_counters - int64_t{1}) * kSlotFloats, a.status);
        };
        auto store_part = [&](float *slot, int r, int d, float4 x, float top, float sum) {
            if (!in_slots(slot)) return;
            *reinterpret_cast<float4 *>(slot + r * kDim + d) = x;
            if (d == 0) slot[kRows * 128 + r] = top, slot[kRows * 128 + kRows + r] = sum;
        };
        // part c of this (sequence, head) lies in the first slot of its CTA, or in the second one where that
        // CTA's range began before the head
        const int c0 = static_cast<int>(share.owner(i0 + kSetup)), parts = static_cast<int>(share.owner(i0 + sp.units - 1)) - c0 + 1;
        const int id0 = 2 * c0 + (share.begin(c0) >= i0 ? 0 : 1);
        auto id_of = [&](int c) { return c ? 2 * (c0 + c) : id0; };
        auto slot_of = [&](int c) { return a.parts + id_of(c) * static_cast<int64_t>(kSlotFloats); };
        for (int i = tid; i < rows * (kDim / 4); i += kThreads) {
            const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
            float top = s_m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(s_m[w][r] - base);
                const float4 y = *reinterpret_cast<const float4 *>(merge + (w * kUsed + r) * kStride + d);
                sum = fmaf(s_l[w][r], f, sum);
                x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
            }
            if (whole) finish(r, d, x, top, sum);
            else store_part(slot_of(blockIdx.x - c0), r, d, x, top, sum);
        }
        // Join of the parts: eight neighbours by the last of them to arrive, then eight of these, and so on;
        // which parts meet is fixed, so the result does not depend on who was last.
        int index = blockIdx.x - c0, stride = 1;
        for (int level = 0; !whole; ++level) {
            const int left = (parts + stride - 1) / stride;  // parts of this level
            if (left == 1) break;
            const int lead = index / kFan * kFan, count = min(kFan, left - lead);
            __syncthreads();  // this CTA's part is written; the fence below publishes it for all threads
            if (tid == 0) {
                const int id = id_of(lead * stride);
                s_last = 0;
                if (in_bounds(level < kLevels && id >= 0 && id < a.level_counters, a.status)) {
                    int32_t *ctr = a.counters + level * a.level_counters + id;
                    int before;
                    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(ctr) : "memory");
                    s_last = before == count - 1;
                    if (s_last) *ctr = 0;  // ready for the next call
                }
            }
            __syncthreads();
            if (!s_last) break;
            if (tid < kFan * kRows) {
                const int q = tid / kRows, r = tid % kRows;
                const bool on = q < count && r < rows && in_slots(slot_of((lead + q) * stride));
                const float *slot = slot_of((lead + (on ? q : 0)) * stride) + kRows * 128;
                s_jm[q][r] = on ? __ldcg(slot + r) : -INFINITY;
                s_jl[q][r] = on ? __ldcg(slot + kRows + r) : 0.f;
            }
            constexpr int kEach = kUsed * (kDim / 4) / kThreads;  // column quadruples of a thread
#pragma unroll
            for (int e = 0; e < kEach; e += 2) {
                float4 y[2][kFan];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int i = tid + (e + w) * kThreads;
#pragma unroll
                    for (int q = 0; q < kFan; ++q)
                        if (e + w < kEach && q < count && i < rows * (kDim / 4) && in_slots(slot_of((lead + q) * stride)))
                            y[w][q] = __ldcg(reinterpret_cast<const float4 *>(slot_of((lead + q) * stride)) + i);
                }
                __syncthreads();
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int i = tid + (e + w) * kThreads;
                    if (e + w >= kEach || i >= rows * (kDim / 4)) continue;
                    const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
                    float top = s_jm[0][r];
#pragma unroll
                    for (int q = 1; q < kFan; ++q) top = fmaxf(top, s_jm[q][r]);
                    const float base = top == -INFINITY ? 0.f : top;
                    float sum = 0.f;
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int q = 0; q < kFan; ++q) {
                        if (q >= count) continue;
                        const float f = ex2(s_jm[q][r] - base);
                        sum = fmaf(s_jl[q][r], f, sum);
                        x.x = fmaf(y[w][q].x, f, x.x), x.y = fmaf(y[w][q].y, f, x.y);
                        x.z = fmaf(y[w][q].z, f, x.z), x.w = fmaf(y[w][q].w, f, x.w);
                    }
                    if (left <= kFan) finish(r, d, x, top, sum);
                    else store_part(slot_of(lead * stride), r, d, x, top, sum);  // in place of the first of the eight
                }
            }
            index /= kFan;
            stride *= kFan;
        }
        __syncthreads();  // shared memory is free again
        }
        at = stop;
        if (!alone && ++vh == vheads && at < end) {
            vh = 0;
            units_before += sp.units;
            do sp = span_of<kBlock>(a, ++b);
            while (sp.units == 0);
        }
    }
}
// Sequences with nothing to see.
template <int kDim, int kBlock>
__device__ __forceinline__ void clear_unseen(const AttnArgs &a) {
    for (int64_t b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
        if (span_of<kBlock>(a, b).units != 0) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + b * a.q_heads * (kDim * 2));
        for (int i = threadIdx.x; i < a.q_heads * (kDim / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int i = threadIdx.x; i < a.q_heads; i += kThreads) a.lse[b * a.q_heads + i] = -INFINITY;
    }
}

// Each warp takes whole heads.
template <int kDim, bool kE4m3, bool kPack>
__global__ void __launch_bounds__(kThreads, kCtasOf<kPack>) attention_alone_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_trigger_and_wait();
    clear_unseen<kDim, kBlockOf<kE4m3>>(a);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    stream<kDim, kE4m3, kPack, true>(a, smem, Share(0, 0), first, static_cast<int64_t>(a.n_seqs) * a.kv_heads * a.subs, 0, 0);
}

template <int kDim, bool kE4m3, bool kPack>
__global__ void __launch_bounds__(kThreads, kCtasOf<kPack>) attention_kernel(const AttnArgs a) {
    constexpr int kBlock = kBlockOf<kE4m3>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[kWarps];
    __shared__ int64_t s_found[2];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int vheads = a.kv_heads * a.subs;
    pdl_trigger_and_wait();

    clear_unseen<kDim, kBlock>(a);

    // all units of work, and this CTA's range of them
    int64_t mine = 0;
    for (int64_t b = tid; b < a.n_seqs; b += kThreads) mine += span_of<kBlock>(a, b).units;
    const int64_t upto = warp_scan(mine);
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    const Share share(static_cast<uint64_t>(s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) * vheads, gridDim.x);
    if (blockIdx.x >= share.ctas) return;
    const int64_t begin = share.begin(blockIdx.x), end = share.begin(blockIdx.x + 1);

    // the sequence that holds unit `begin`, and the units before it
    if (a.n_seqs <= kThreads) {  // one sequence per thread: the sums above are the positions
        int64_t p = upto - mine;
        for (int w = 0; w < warp; ++w) p += s_sum[w];
        if (mine > 0 && p * vheads <= begin && begin < (p + mine) * vheads) s_found[0] = tid, s_found[1] = p;
    } else {
        int64_t before = 0;
        for (int64_t b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
            __syncthreads();
            const int64_t n = b0 + tid < a.n_seqs ? span_of<kBlock>(a, b0 + tid).units : 0;
            const int64_t in = warp_scan(n);
            if (lane == 31) s_sum[warp] = in;
            __syncthreads();
            int64_t p = before + in - n;
            for (int w = 0; w < warp; ++w) p += s_sum[w];
            if (n > 0 && p * vheads <= begin && begin < (p + n) * vheads) s_found[0] = b0 + tid, s_found[1] = p;
            before += s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
        }
    }
    __syncthreads();
    stream<kDim, kE4m3, kPack, false>(a, smem, share, begin, end, s_found[0], s_found[1]);
}

template <int kDim, bool kE4m3, bool kPack, bool alone>
cudaError_t launch_form(const AttnArgs &a, const DevCtx &ctx, cudaStream_t stream) {
    constexpr int smem_size = smem_bytes<kDim, kE4m3>();
    constexpr auto kernel = alone ? attention_alone_kernel<kDim, kE4m3, kPack> : attention_kernel<kDim, kE4m3, kPack>;
    const cudaError_t e = allow_smem<kernel>(smem_size, ctx.device);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctx.num_sms * kCtasOf<kPack>));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_size;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kDim, bool kE4m3, bool kPack>
cudaError_t launch_typed(const AttnArgs &a, const DevCtx &ctx, cudaStream_t stream) {
    // The host has no lengths, but the page table's width and the window bound them.  With few keys to a head a CTA's
    // steps are mostly its setup and joins, so each warp takes heads by itself where that is not many more steps and no
    // head can have more than kAloneKeys keys: beyond that one long sequence among short ones keeps its few warps busy
    // alone (224 sequences, 8 KV heads, one of 65536 tokens, the others of 64: 59 us split, 2254 alone).  By CTAs and by
    // warps, 32 and 8 heads, bf16, us, all sequences as long as the table allows / lengths spread in their logarithm:
    //   200 sequences up to  64: 15.5, 8.1 / 14.7, 7.1;   256: 42.5, 36.2 / 18.7, 13.8;  512: 71.0, 65.3 / 21.4, 22.4
    //                      4096: 487, 482 / -;           8191: - / 121, 308
    //   64 sequences up to   64: 8.3, 6.7 / 8.0, 6.2;     192: 13.2, 12.5 / 10.8, 10.4;  256: 14.6, 15.2 / 10.8, 12.2
    const int64_t width = static_cast<int64_t>(a.max_pages) * a.page_size;
    const int64_t keys = a.window > 0 ? std::min<int64_t>(width, a.window) : width;  // that a query may see,
    const int64_t most = a.window > 0 ? std::min<int64_t>(width, keys + kTileOf<kE4m3> - 1) : width;  // and with what else their tiles hold
    const int64_t heads = static_cast<int64_t>(a.n_seqs) * a.kv_heads * a.subs, ctas = ctx.num_sms * kCtasOf<kPack>;
    const int64_t tiles = (most + kTileOf<kE4m3> - 1) / kTileOf<kE4m3>, blocks = (tiles + kWarps - 1) / kWarps;
    const int64_t steps = (heads * (blocks + kSetup) + ctas - 1) / ctas;
    const int64_t steps_alone = (heads + ctas * kWarps - 1) / (ctas * kWarps) * (tiles + kSetup);
    if (keys <= kAloneKeys && steps_alone <= steps + steps / 4 + 5) return launch_form<kDim, kE4m3, kPack, true>(a, ctx, stream);
    return launch_form<kDim, kE4m3, kPack, false>(a, ctx, stream);
}

int slots_of(int num_sms) { return 2 * num_sms * kMaxCtasPerSm; }
size_t part_bytes(int num_sms) { return static_cast<size_t>(slots_of(num_sms)) * kSlotFloats * sizeof(float); }

int subs_of(int group) { return (group + kRows - 1) / kRows; }

}  // namespace

// Slots and counters belong to CTAs, so the workspace has one size for every batch.
size_t attention_workspace_size(int num_sms) {
    return part_bytes(num_sms) + (static_cast<size_t>(kLevels) * slots_of(num_sms) * sizeof(int32_t) + 255) / 256 * 256;
}

cudaError_t launch_attention(const bd_kv_cache &c, const void *q, int32_t q_heads, const int32_t *page_table,
                             const int32_t *lengths, int32_t n_seqs, int32_t max_pages, float scale, int32_t window,
                             void *out, float *lse, void *workspace, const DevCtx &ctx, cudaStream_t stream) {
    AttnArgs a;
    a.q = static_cast<const uint8_t *>(q);
    a.ck = static_cast<const uint8_t *>(c.k);
    a.cv = static_cast<const uint8_t *>(c.v);
    a.ck_scale = c.k_scale;
    a.cv_scale = c.v_scale;
    a.page_table = page_table;
    a.lengths = lengths;
    a.out = static_cast<uint8_t *>(out);
    a.lse = lse;
    a.parts = static_cast<float *>(workspace);
    a.counters = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + part_bytes(ctx.num_sms));
    a.level_counters = slots_of(ctx.num_sms);
    a.status = ctx.status;
    a.n_pages = c.n_pages;
    a.n_seqs = n_seqs;
    a.max_pages = max_pages;
    a.kv_heads = c.kv_heads;
    a.page_size = c.page_size;
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.subs = subs_of(a.group);
    a.window = window;
    a.page_tiles = static_cast<uint32_t>(c.page_size / 16);
    // exact while piece * (page_tiles - 1) < 2^32: pieces stay below 2^26, page_tiles at most 64
    a.page_magic = static_cast<uint32_t>(((uint64_t{1} << 32) + a.page_tiles - 1) / a.page_tiles);
    a.scale_log2 = scale * 1.44269504088896f;
    const bool e = c.kv_type == BD_KV_E4M3, pack = a.group <= 8;
    if (c.head_dim == 128) {
        if (e) return pack ? launch_typed<128, true, true>(a, ctx, stream) : launch_typed<128, true, false>(a, ctx, stream);
        return pack ? launch_typed<128, false, true>(a, ctx, stream) : launch_typed<128, false, false>(a, ctx, stream);
    }
    if (e) return pack ? launch_typed<64, true, true>(a, ctx, stream) : launch_typed<64, true, false>(a, ctx, stream);
    return pack ? launch_typed<64, false, true>(a, ctx, stream) : launch_typed<64, false, false>(a, ctx, stream);
}

}  // namespace bd
