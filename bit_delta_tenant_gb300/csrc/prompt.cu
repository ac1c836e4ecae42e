// prompt.cu -- attention of prompts over a paged key-value cache, on the tensor cores.
//
//   o = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),  s_j the score rule of q . K_j
//
// Bound: tensor cores (4 head_dim products per seen pair, and 2 head_dim for the second parts of its weights; a block of 128 keys against
// 256 rows is 1.5 x 2048 clocks of tcgen05 at head_dim 128, its 32768 exponentials about a third of that), HBM or latency for a few queries.
//
// Work.  A row is one query of one head; the heads that share a KV head are rows of the same tile, so that K and V are
// read once for all of them and a tile of 128 rows holds 128 / heads tokens.  A unit is two such tiles (256 rows) of
// one sequence and KV head, or, where units are fewer than SMs, a piece of its keys; each CTA (one per SM) takes the next
// unit when it has finished one, those of most keys first.  Pieces leave their unnormalised output, maximum and sum in
// the workspace and a second kernel joins them in key order, so results do not depend on timing.
//
// A CTA.  Warps 0-3 and 4-7: the softmax of one tile each, a thread per row.  Warp 8: issues the products.  Warp 9: finds
// the next unit and its blocks.  Warp 10 on: K and V of the cache to a ring of shared-memory tiles, by TMA in
// bf16 (warp 10; warp 11 looks at the blocks that some row sees only in part); 8-bit and 4-bit values are copied as they are and
// converted by warps 11 to 15.
// S = Q K^T goes to tensor memory; a softmax thread reads its row, and writes the weights back there as 16-bit operands of
// P V, whose accumulator stays in tensor memory.  The two tiles alternate: one's products run under the other's softmax.
// A weight is a 16-bit number and the 16-bit rest, two products, so that no more is lost than in single tokens' attention: 2^-16 of it
// (one bf16 number: 2^-8, outputs off by 2.2e-3 where their own rounding is 1.6e-3, 8192 tokens in 391 us instead of 521).
// The running maximum is raised only when a row passes it by 2^8 (4 bits: 2^3), so that the output is seldom rescaled:
// weights are at most that, sums stay fp32.
//
// Values that a row does not see.  A weight of 0 does not hide an infinity or NaN of V.  Blocks that some row sees in part
// are looked at: rows of V that nobody sees are zeroed, and where a finite number is missing in another one, the
// block's P V is added up by the softmax threads, row by row over the keys that the row sees, instead of by the tensor cores.
//
// Measured (head_dim 128, 32 and 8 heads unless said): one prompt of 8192 tokens, bf16, 485 us in short runs, 521 at the power cap (1.13
// and 1.06 PFLOP/s without the second parts' products, 1.7 and 1.6 with them): a block takes about 3800 clocks, its products 1.5 x 2048; a
// tile's softmax and its own products follow each other, and the thread that issues them shares its scheduler with two softmax warps.
// 333 tokens 17.8 us: launch, set-up, three blocks one after the other, output.  Over 8 and 4 bits the 64 KB that are stored to shared
// memory for a block contend with the products' reads of their operands (8192 tokens 621 and 728 us; 48 tokens over 65000, 64 and 8 heads: bf16
// 140 us, 8 bits 180, 4 bits 200).  Caps cost a pass of their own over the scores, with an exponential where they are not small: 9 ragged
// prompts of up to 1500 tokens over up to 1000, 8 bits, 84 us, 59 uncapped.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "bd_device.cuh"
#include "bd_internal.h"
#include "bd_rows.cuh"

namespace bd {
namespace {

constexpr int kBlock = 128;  // keys of a block
constexpr int kTileRows = 128;
constexpr int64_t kMaxLength = 1 << 30;
constexpr int kConvertWarps = 5;
// A 4-bit cache's values over 8 are fp16 numbers, whatever their scale, and take two operations a pair to make, bf16 ones five:
// its products are of fp16, Q turned to fp16 in shared memory, each row times a power of two of its own, and the weights
// times 2^kLift, so that small ones are kept (two parts are off by 2^-22 of a weight, or by 2^-37 of the largest).
template <int kType>
constexpr bool kHalf = kType == BD_KV_E2M1;
template <int kType>
constexpr float kLift = kHalf<kType> ? 12.f : 0.f;
template <int kType>
constexpr float kLazy = kHalf<kType> ? 3.f : 8.f;  // by how much (in base 2) a row's scores may pass the maximum they are taken from

template <int kType>
constexpr int kThreadsOf = kType == BD_KV_BF16 ? 384 : 512;
template <int kDim>
constexpr uint32_t kTileBytes = kBlock * kDim * 2;  // of K, V or Q in shared memory: columns in pieces of 64, swizzled
// K and V tiles in shared memory; 8 and 4 bits: and tiles as they are in the cache, with their scale bytes behind the values
template <int kDim, int kType>
constexpr int kStages = kDim == 128 ? (kType == BD_KV_BF16 ? 5 : 4) : (kType == BD_KV_BF16 ? 8 : 6);
template <int kDim, int kType>
constexpr int kRow = kType == BD_KV_BF16 ? 2 * kDim : kType == BD_KV_E4M3 ? kDim : kDim / 2;  // bytes of a key
template <int kDim, int kType>
constexpr int kScale = kType == BD_KV_BF16 ? 0 : kType == BD_KV_E4M3 ? 1 : kDim / 16;
template <int kDim, int kType>
constexpr int kRawSlots = kType == BD_KV_BF16 ? 0 : kDim == 64 ? 4 : kType == BD_KV_E4M3 ? 2 : 3;
template <int kDim, int kType>
constexpr int kRawBytes = kBlock * (kRow<kDim, kType> + kScale<kDim, kType>);
template <int kDim, int kType>
constexpr int kSmemBytes = 1024 + (2 + kStages<kDim, kType>) * kTileBytes<kDim> + kRawSlots<kDim, kType> * kRawBytes<kDim, kType> + 1024;
constexpr int kSlotRows = 2 * kTileRows;
template <int kDim>
constexpr int64_t kSlotFloats = kSlotRows * (kDim + 2);  // a piece's output, maxima and sums, tile by tile

// A unit: tokens row0 .. of q (positions pos0 ..) against blocks blk0 .. of the sequence's keys.
struct Unit {
    int32_t seq, row0, tokens, pos0, len, prefix, vh;
    int32_t blk0, blocks;  // blocks < 0: no more units
    int32_t in_lo, in_hi;  // keys that every row that sees any sees
    int32_t un_lo, un_hi;  // keys that some row sees
    int32_t slot, parts;   // a piece's slot and how many there are, or -1 and 1
    int32_t state;         // kFirstPiece; kGaps: some page id is out of range
};
constexpr int kFirstPiece = 1, kGaps = 2;
static_assert(sizeof(Unit) == 64);

struct PromptArgs {
    const uint8_t *ck, *cv, *ck_scale, *cv_scale;
    const int32_t *page_table, *offsets, *lengths, *first, *prefix;
    const float *slopes;
    uint8_t *out;
    float *lse, *parts;
    unsigned *taken;  // units taken, and CTAs that take no more
    int4 *heads;  // of the joining kernel: per slot, {pieces, first row of q, tokens, KV head} of a unit's first piece
    unsigned *status;
    uint64_t wait_ns;
    int64_t n_pages, total;
    int32_t n_seqs, max_pages, page_size, kv_heads, q_heads;
    int32_t group, subs, heads_tile, tile_tokens;  // query heads of a KV head, in `subs` lots of heads_tile; tokens of a tile
    int32_t window, slots, box;                    // box: keys of one TMA copy
    float scale_log2, cap, cap_in;
    int32_t may_split, plain;                      // plain: scores are products times a positive scale
    float v_unit;                                  // what V is given over
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t bits_of(float2 v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 pair_of(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits_of(x)), "l"(bits_of(y)), "l"(bits_of(z)));
    return pair_of(r);
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(x)), "l"(bits_of(y)));
    return pair_of(r);
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(x)), "l"(bits_of(y)));
    return pair_of(r);
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ float tmem_ld_one(uint32_t taddr) {
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
    tmem_ld_wait();
    return __uint_as_float(v);
}
// Byte of 16-byte chunk c (8 columns) of row r in a tile: pieces of 64 columns, chunks turned by the row.
__device__ __forceinline__ uint32_t tile_at(int r, int c) { return (c / 8) * (kBlock * 128) + r * 128 + (((c % 8) ^ (r & 7)) << 4); }

// 0 times each of a bf16 pair, added to `sum`: NaN from an infinity or NaN on.
__device__ __forceinline__ uint32_t zero_times(uint32_t pair, uint32_t sum) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(pair), "r"(0u), "r"(sum));
    return r;
}
__device__ __forceinline__ uint32_t half2_times(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t byte) {  // the low byte's two values
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(byte));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool half>
__device__ __forceinline__ float2 unpack_pair(uint32_t pair) {
    if constexpr (half) return __half22float2(*reinterpret_cast<const __half2 *>(&pair));
    else return make_float2(bf16lo_to_f32(pair), bf16hi_to_f32(pair));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

struct Smem {
    uint64_t *full, *empty, *fixed;      // per stage
    uint64_t *raw_full, *raw_empty;      // per slot of tiles as they are in the cache
    uint8_t *raw;
    uint64_t *q_full, *q_ready, *q_empty, *s_full, *p_full, *o_full;  // per tile
    uint64_t *u_full, *u_empty;          // per unit slot
    uint64_t *u_want;                    // warp 10 is ready for the next unit
    Unit *unit;
    volatile int *slow;                  // per stage: number (from 1) of the last load of a V that is not finite and not seen by all
    volatile int *abort;
    uint32_t *tmem;
};

// Bounded wait of one thread; on give-up the status word and the other roles are told.
__device__ __forceinline__ bool wait_alone(uint64_t *bar, uint32_t parity, const PromptArgs &a, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    if (a.wait_ns != 0) {
        // the clock and the flag are looked at seldom: most waits are over sooner than they are read
        uint64_t begin = 0;
        for (int polls = 1;; ++polls) {
            if (mbar_try_wait(bar, parity)) return true;
            if (polls % 64) continue;
            const uint64_t now = globaltimer_ns();
            if (begin == 0) begin = now;
            if (*abort != 0 || now - begin > a.wait_ns) break;
        }
    }
    *abort = 1;
    flag_status(a.status, kDevTimeout);
    return false;
}
// The same of a warp.
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, const PromptArgs &a, volatile int *abort) {
    return __all_sync(0xFFFFFFFFu, wait_alone(bar, parity, a, abort));
}

// ---- units -----------------------------------------------------------------------------

struct Sequence {
    int32_t row0, n, len, prefix;
    int32_t units, blocks;  // of a KV head: tiles' pairs, and blocks of the longest
};
// `ordered`: false where its offsets are no rows of q.
__device__ __forceinline__ Sequence sequence_of(const PromptArgs &a, int64_t i, bool &ordered) {
    Sequence s = {};
    const int32_t from = a.offsets[i], to = a.offsets[i + 1];
    const int64_t most = min(static_cast<int64_t>(a.max_pages) * a.page_size, kMaxLength);
    int64_t len = a.lengths[i];
    ordered = from >= 0 && to >= from && to <= a.total;
    if (!ordered || len < 0 || len > most || (i == 0 && from != 0)) flag_status(a.status, kDevBadIndex);
    len = len < 0 ? 0 : len > most ? most : len;
    s.len = static_cast<int32_t>(len);
    if (!ordered) return s;
    s.row0 = from;
    s.n = to - from;
    if (s.n > s.len) flag_status(a.status, kDevBadIndex);
    s.prefix = a.prefix ? max(0, min(a.prefix[i], s.len)) : 0;
    const int pair = 2 * a.tile_tokens;
    s.units = (s.n + pair - 1) / pair;
    s.blocks = (s.len + kBlock - 1) / kBlock;
    if (a.window > 0) s.blocks = static_cast<int32_t>(min(static_cast<int64_t>(s.blocks), (static_cast<int64_t>(a.window) + max(pair, s.prefix)) / kBlock + 2));
    return s;
}
__device__ __forceinline__ int32_t pieces_of(const Sequence &s, int32_t most) { return s.blocks > most ? (s.blocks + most - 1) / most : 1; }

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ int64_t warp_scan(int64_t v) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (static_cast<int>(threadIdx.x % 32) >= o) v += u;
    }
    return v;
}

// A pass over the sequences, 32 at a time, a lane each.  Sequences that begin before an offset that came earlier are left out, so that no two
// have a row in common.
struct Pass {
    bool disorder = false;
    int32_t top = INT_MIN;  // of the offsets so far, from the first disorder on
    __device__ __forceinline__ Sequence take(const PromptArgs &a, int64_t i) {
        Sequence s = {};
        bool ordered = true;
        if (i < a.n_seqs) s = sequence_of(a, i, ordered);
        disorder |= __any_sync(0xFFFFFFFFu, !ordered);
        if (disorder) {  // until now the offsets ascended to this lot's first
            const int32_t from = i < a.n_seqs ? a.offsets[i] : INT_MIN;
            int32_t most = from;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int32_t u = __shfl_up_sync(0xFFFFFFFFu, most, o);
                if (static_cast<int>(threadIdx.x % 32) >= o) most = max(most, u);
            }
            most = max(most, top);
            if (from < most) s = Sequence{};
            top = __shfl_sync(0xFFFFFFFFu, most, 31);
        }
        return s;
    }
};

__device__ __forceinline__ int size_class(const Sequence &q) { return q.units > 0 ? 31 - __clz(max(q.blocks, 1)) : -1; }

// Warp 9.  Units are numbered sequence by sequence, those of most keys first by powers of two, in each from its last tile to
// its first (then pieces, then KV heads): whoever takes the next unit takes one of the largest that are left.
__device__ __forceinline__ void find_units(const PromptArgs &a, const Smem &s) {
    const int lane = threadIdx.x % 32;
    const int vheads = a.kv_heads * a.subs, pair = 2 * a.tile_tokens;
    // blocks of a piece: as few as give every CTA a unit at most, where whole units leave CTAs without one
    int32_t most = 1 << 30;
    unsigned classes = 0;
    int64_t units = 0, blocks = 0;
    Sequence q = {};
    Pass pass;
    for (int64_t i = lane; i - lane < a.n_seqs; i += 32) {
        q = pass.take(a, i);
        if (q.units > 0) classes |= 1u << size_class(q);
        units += q.units, blocks += static_cast<int64_t>(q.units) * q.blocks;
    }
    classes = __reduce_or_sync(0xFFFFFFFFu, classes);
    if (a.may_split) {
        units = warp_sum(units) * vheads, blocks = warp_sum(blocks) * vheads;
        if (units <= a.slots) {
            most = max(4, static_cast<int32_t>((blocks + a.slots - 1) / a.slots));
            while (true) {
                int64_t pieces = 0;
                pass = Pass{};
                for (int64_t i = lane; i - lane < a.n_seqs; i += 32) {
                    if (a.n_seqs > 32) q = pass.take(a, i);
                    pieces += static_cast<int64_t>(q.units) * pieces_of(q, most);
                }
                if (warp_sum(pieces) * vheads <= a.slots) break;
                most += most / 16 + 1;
            }
        }
    }
    int64_t first = a.n_seqs, before = 0;  // the 32 sequences looked at, and the units of those before them
    int cls = 32;
    int64_t mine = 0, upto = 0, all = 0;
    auto look = [&] {  // at the next sequences; false: there are none
        before += all;
        first += 32;
        if (first >= a.n_seqs) {
            classes &= cls < 32 ? (1u << cls) - 1 : 0xFFFFFFFFu;
            if (classes == 0) return false;
            cls = 31 - __clz(classes);
            first = 0;
            pass = Pass{};
        }
        if (a.n_seqs > 32) q = pass.take(a, first + lane);  // else each lane has its own still
        mine = size_class(q) == cls ? static_cast<int64_t>(q.units) * pieces_of(q, most) * vheads : 0;
        upto = warp_scan(mine);
        all = __shfl_sync(0xFFFFFFFFu, upto, 31);
        return true;
    };
    bool over = false;
    int it = 0;
    for (int64_t round = 0; !over; ++round) {
        // Where units are split there are no more than CTAs, and CTA b takes unit b, whose slot is b.  The host, which has no lengths, also
        // says that they may be split for batches of short pieces that make more units than CTAs: none is split then, and CTAs take
        // them in turn.  Else the next one, taken when warp 10 has started the last copies of the one before: a unit taken
        // earlier waits here while other CTAs run dry.
        if (!wait_on(s.u_want, it & 1, a, s.abort)) break;
        int64_t u = round * gridDim.x + blockIdx.x;
        if (!a.may_split) u = __shfl_sync(0xFFFFFFFFu, lane == 0 ? atomicAdd(a.taken, 1u) : 0u, 0);
        while (!over && u >= before + all) over = !look();
        Unit d = {};
        d.blocks = -1;
        if (!over) {
            const unsigned holds = __ballot_sync(0xFFFFFFFFu, u < before + upto);
            const int owner = __ffs(holds) - 1;  // the first whose units reach beyond u
            int64_t at = u - before - __shfl_sync(0xFFFFFFFFu, upto - mine, owner);
            Sequence w;
            w.row0 = __shfl_sync(0xFFFFFFFFu, q.row0, owner), w.n = __shfl_sync(0xFFFFFFFFu, q.n, owner);
            w.len = __shfl_sync(0xFFFFFFFFu, q.len, owner), w.prefix = __shfl_sync(0xFFFFFFFFu, q.prefix, owner);
            w.units = __shfl_sync(0xFFFFFFFFu, q.units, owner), w.blocks = __shfl_sync(0xFFFFFFFFu, q.blocks, owner);
            const int pieces = pieces_of(w, most);
            d.seq = static_cast<int32_t>(first + owner);
            d.vh = static_cast<int32_t>(at % vheads);
            at /= vheads;
            const int piece = static_cast<int>(at % pieces);
            const int tile = w.units - 1 - static_cast<int>(at / pieces);
            d.row0 = w.row0 + tile * pair;
            d.tokens = min(pair, w.n - tile * pair);
            d.pos0 = w.len - w.n + tile * pair;
            d.len = w.len, d.prefix = w.prefix;
            // what its rows see
            int un_lo = INT_MAX, un_hi = 0, in_lo = 0, in_hi = INT_MAX;
            for (int t = lane; t < d.tokens; t += 32) {
                const int p = d.pos0 + t;
                if (p < 0) continue;
                const int hi = max(p + 1, d.prefix);
                int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
                if (a.first && in_bounds(d.row0 + t < a.total, a.status)) lo = max(lo, a.first[d.row0 + t]);
                if (lo >= hi) continue;
                un_lo = min(un_lo, lo), un_hi = max(un_hi, hi), in_lo = max(in_lo, lo), in_hi = min(in_hi, hi);
            }
            un_lo = __reduce_min_sync(0xFFFFFFFFu, un_lo), un_hi = __reduce_max_sync(0xFFFFFFFFu, un_hi);
            in_lo = __reduce_max_sync(0xFFFFFFFFu, in_lo), in_hi = __reduce_min_sync(0xFFFFFFFFu, in_hi);
            int b0 = 0, b1 = 0;
            if (un_lo < un_hi) b0 = un_lo / kBlock, b1 = (un_hi + kBlock - 1) / kBlock;
            d.slot = -1, d.parts = 1;
            if (pieces > 1) {
                const int whole = b1 - b0, parts = max(1, (whole + most - 1) / most);
                if (piece >= parts) continue;  // shorter than the sequence's longest
                if (parts > 1) d.slot = static_cast<int32_t>(u), d.parts = parts;
                b0 += piece * most;
                b1 = min(b1, b0 + most);
            }
            d.blk0 = b0, d.blocks = b1 - b0;
            d.in_lo = in_lo, d.in_hi = in_hi, d.un_lo = un_lo, d.un_hi = un_hi;
            d.state = piece == 0 ? kFirstPiece : 0;
            const int32_t *table = a.page_table + static_cast<int64_t>(d.seq) * a.max_pages;
            bool gaps = false;
            const int key0 = max(un_lo, b0 * kBlock), key1 = min(un_hi, b1 * kBlock);
            if (key0 < key1) {
                const int last = (key1 - 1) / a.page_size;
#pragma unroll 4
                for (int i = key0 / a.page_size + lane; i <= last; i += 32)
                    if (in_bounds(i < a.max_pages, a.status)) gaps |= table[i] < 0 || table[i] >= a.n_pages;
            }
            if (__any_sync(0xFFFFFFFFu, gaps)) d.state |= kGaps;
        }
        if (!wait_on(&s.u_empty[it & 1], ((it >> 1) & 1) ^ 1, a, s.abort)) break;
        if (lane == 0) {
            s.unit[it & 1] = d;
            mbar_arrive(&s.u_full[it & 1]);
        }
        __syncwarp();
        ++it;
    }
    // the last CTA to have taken all it takes leaves the count ready for the next call
    if (!a.may_split && lane == 0 && atomicAdd(a.taken + 1, 1u) == gridDim.x - 1) a.taken[0] = a.taken[1] = 0;
}

// The next unit, or blocks < 0 after the last one and on give-up.
__device__ __forceinline__ Unit next_unit(const PromptArgs &a, const Smem &s, int &it) {
    Unit u;
    u.blocks = -1;
    if (!wait_on(&s.u_full[it & 1], (it >> 1) & 1, a, s.abort)) return u;
    u = s.unit[it & 1];
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&s.u_empty[it & 1]);
    ++it;
    return u;
}

__device__ __forceinline__ bool seen_in_part(const Unit &u, int blk) { return blk * kBlock < u.in_lo || (blk + 1) * kBlock > u.in_hi; }

// ---- warp 8: products --------------------------------------------------------------------

extern __shared__ uint8_t smem_raw[];
__device__ __forceinline__ uint32_t smem_base() { return (smem_u32(smem_raw) + 1023u) & ~1023u; }

// Tensor memory is allocated whole, so its columns are counted from 0: S of the tiles, then O of the tiles.  The weights take the
// place of the scores that they are made of: for each 16 keys 8 columns of first parts, 8 of second parts.
constexpr uint32_t kColS = 0, kColO = 2 * kBlock;
__device__ __forceinline__ constexpr uint32_t weight_at(int key) { return key / 16 * 16 + key % 16 / 2; }  // second part: + 8

// The products with a descriptor's lower word given: its upper word is one for all tiles, and one addition a product is left.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;  // 1024 bytes to the next 8 rows, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t leading) { return (addr & 0x3FFFFu) >> 4 | (leading >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
template <int kType>
constexpr uint32_t idesc_of(int n) { return idesc_bf16_f32(kTileRows, n) & ~(kHalf<kType> ? 1u << 7 | 1u << 10 : 0u); }
// S of a tile: Q K^T.
template <int kDim, int kType, int kTile>
__device__ __forceinline__ void issue_scores(int stage) {
    constexpr uint32_t idesc = idesc_of<kType>(kBlock);
    const uint32_t q = desc_low(smem_base() + kTile * kTileBytes<kDim>, 16), k = desc_low(smem_base() + (2 + stage) * kTileBytes<kDim>, 16);
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) {
        const uint32_t at = i / 4 * (kBlock * 128 / 16) + i % 4 * 2;
        mma_ss(kColS + kTile * kBlock, q + at, k + at, idesc, i > 0);
    }
}
// Half of a tile's P V, each 16 keys' first and second parts; V's rows are the product's inner dimension, its next 64 columns a
// column piece further.
template <int kDim, int kType, int kTile, int kPart>
__device__ __forceinline__ void issue_values(int stage, uint32_t accumulate) {
    constexpr uint32_t idesc = idesc_of<kType>(kDim) | 1u << 16;
    const uint32_t v = desc_low(smem_base() + (2 + stage) * kTileBytes<kDim>, kBlock * 128);
#pragma unroll
    for (int i = kPart * (kBlock / 32); i < (kPart + 1) * (kBlock / 32); ++i)
#pragma unroll
        for (int second = 0; second < 2; ++second)
            mma_ts(kColO + kTile * kDim, kColS + kTile * kBlock + weight_at(i * 16) + second * 8, v + i * (16 * 128 / 16), idesc,
                   i + second > 0 ? 1u : accumulate);
}

// Run by one thread.  Issuing a product stalls while a few are queued, so this thread's time is the tensor cores': with eight
// softmax warps competing for the schedulers each instruction of it counts (a warp that elects a lane for each lot of
// products took 137 clocks a product beside busy warps, one thread throughout 90, a thread chosen by its number 275).
template <int kDim, int kType>
__device__ __forceinline__ void issue_products(const PromptArgs &a, const Smem &s) {
    constexpr int kS = kStages<kDim, kType>;
    int it = 0;
    uint32_t p_round[2] = {0, 0}, q_round[2] = {0, 0};
    uint32_t o_round[2] = {1, 1};  // of a tile's last products; there are none yet
    int stage = 0, loads = 0;
    uint32_t round = 0;  // of the next K or V tile
    bool ok = true;
    auto advance = [&] {
        ++loads;
        if (++stage == kS) stage = 0, round ^= 1;
    };
    std::integral_constant<int, 0> first;
    std::integral_constant<int, 1> second;
    int blocks = 0, blk0 = 0, in_lo = 0, in_hi = 0;
    bool both = false;
    auto next = [&] {  // the next unit with something to see; false: none
        do {
            if (!wait_alone(&s.u_full[it & 1], (it >> 1) & 1, a, s.abort)) return false;
            const Unit &u = s.unit[it & 1];
            blocks = u.blocks, blk0 = u.blk0, in_lo = u.in_lo, in_hi = u.in_hi, both = u.tokens > a.tile_tokens;
            mbar_arrive(&s.u_empty[it & 1]);
            ++it;
        } while (blocks == 0);
        return blocks > 0;
    };
    // Scores take the place of the last weights.  Products of one shape run in the order they are issued in; at head_dim 64 the
    // two are of different shapes.
    auto scores_free = [&](auto tile) { return kDim == 128 || wait_alone(&s.o_full[tile()], o_round[tile()], a, s.abort); };
    auto start_tile = [&](auto tile) {
        constexpr int i = tile();
        if (!wait_alone(kHalf<kType> ? &s.q_ready[i] : &s.q_full[i], q_round[i], a, s.abort)) return false;
        q_round[i] ^= 1;
        if (!scores_free(tile)) return false;
        issue_scores<kDim, kType, i>(stage);
        tc_commit(&s.s_full[i]);
        if (blocks == 1) tc_commit(&s.q_empty[i]);
        return true;
    };
    auto start = [&] {  // scores of a unit's first block
        if (!wait_alone(&s.full[stage], round, a, s.abort)) return false;
        if (!start_tile(first)) return false;
        if (both && !start_tile(second)) return false;
        tc_commit(&s.empty[stage]);
        advance();
        return true;
    };
    while (ok && next()) {
        ok = start();
        for (int j = 0; ok && j < blocks; ++j) {
            const int v_stage = stage, key0 = (blk0 + j) * kBlock;
            const uint32_t v_round = round;
            advance();
            const bool part = key0 < in_lo || key0 + kBlock > in_hi, more = j + 1 < blocks;
            ok = wait_alone(kType == BD_KV_BF16 && part ? &s.fixed[v_stage] : &s.full[v_stage], v_round, a, s.abort);
            const bool slow = part && s.slow[v_stage] == loads;  // its load's number from 1
            auto tile_products = [&](auto tile) {
                constexpr int i = tile();
                if (!wait_alone(&s.p_full[2 * i], p_round[i], a, s.abort)) return false;
                tc_fence_after();
                if (!slow) issue_values<kDim, kType, i, 0>(v_stage, j > 0);
                if (!wait_alone(&s.p_full[2 * i + 1], p_round[i], a, s.abort)) return false;
                tc_fence_after();
                p_round[i] ^= 1;
                if (!slow) issue_values<kDim, kType, i, 1>(v_stage, 1);
                tc_commit(&s.o_full[i]);
                o_round[i] ^= 1;
                if (more) {
                    if (i == 0 && !wait_alone(&s.full[stage], round, a, s.abort)) return false;
                    if (!scores_free(tile)) return false;
                    issue_scores<kDim, kType, i>(stage);
                    tc_commit(&s.s_full[i]);
                    if (j + 2 == blocks) tc_commit(&s.q_empty[i]);
                }
                return true;
            };
            ok = ok && tile_products(first) && (!both || tile_products(second));
            if (!ok) break;
            tc_commit(&s.empty[v_stage]);
            if (more) {
                tc_commit(&s.empty[stage]);
                advance();
            }
        }
    }
    // no product may be in flight when tensor memory is freed, even after giving up
    tc_commit(s.o_full + 2);
    mbar_wait(s.o_full + 2, 0, kDrainLimitNs, nullptr);
}

// ---- warp 10 and on: queries, keys and values ------------------------------------------------

template <int kDim>
__device__ __forceinline__ bool load_queries(const PromptArgs &a, const Smem &s, const CUtensorMap *map, uint32_t smem_q, const Unit &u, int (&q_n)[2]) {
    const int tiles = u.tokens > a.tile_tokens ? 2 : 1;
    for (int i = 0; i < tiles; ++i) {
        if (!wait_on(&s.q_empty[i], (q_n[i] & 1) ^ 1, a, s.abort)) return false;
        ++q_n[i];
        if (threadIdx.x % 32 == 0) {
            mbar_arrive_expect_tx(&s.q_full[i], a.heads_tile * a.tile_tokens * kDim * 2);
            const int head = u.vh / a.subs * a.group + u.vh % a.subs * a.heads_tile;
            for (int c = 0; c < kDim / 64; ++c)
                tma_load_3d(smem_q + i * kTileBytes<kDim> + c * (kTileRows * 128), map, &s.q_full[i], c * 64, head, u.row0 + i * a.tile_tokens);
        }
        __syncwarp();
    }
    return true;
}

// Warp 10.  bf16: TMA copies of `box` keys and 64 columns to the tiles; 8 and 4 bits: plain copies of `box` keys and their scale
// bytes.  Lane l looks up piece l of a block and copies it; a piece that no row sees or whose page id is out of range is
// zeroed.
template <int kDim, int kType>
__device__ __forceinline__ void load_tiles(const PromptArgs &a, const Smem &s, const CUtensorMap *map_q, const CUtensorMap *map_k,
                                           const CUtensorMap *map_v, uint32_t smem_q, uint8_t *kv) {
    constexpr bool kCopy = kType != BD_KV_BF16;
    constexpr int kS = kCopy ? kRawSlots<kDim, kType> : kStages<kDim, kType>;
    constexpr int kR = kRow<kDim, kType>, kSc = kScale<kDim, kType>;
    uint64_t *full = kCopy ? s.raw_full : s.full, *empty = kCopy ? s.raw_empty : s.empty;
    const int lane = threadIdx.x % 32;
    const int per_block = kBlock / a.box;
    int it = 0, loads = 0, q_n[2] = {0, 0};
    bool ok = true;
    while (ok) {
        if (lane == 0) mbar_arrive(s.u_want);
        const Unit u = next_unit(a, s, it);
        if (u.blocks < 0) break;
        if (u.blocks == 0) continue;
        const int32_t *table = a.page_table + static_cast<int64_t>(u.seq) * a.max_pages;
        const int kvh = u.vh / a.subs;
        auto page_of = [&](int j) {  // of this lane's piece of block blk0 + j; -1: none
            const int key = (u.blk0 + j) * kBlock + lane * a.box;
            if (lane >= per_block || j >= u.blocks || key >= u.un_hi || key + a.box <= u.un_lo) return -1;
            const int at = key / a.page_size;
            return in_bounds(at >= 0 && at < a.max_pages, a.status) ? table[at] : -1;
        };
        int next_page = page_of(0);
        if (!load_queries<kDim>(a, s, map_q, smem_q, u, q_n)) break;
        for (int j = 0; j < u.blocks && ok; ++j) {
            int page = next_page;
            next_page = page_of(j + 1);  // not waited for until the next block
            const int key = (u.blk0 + j) * kBlock + lane * a.box;
            if (page < 0 || page >= a.n_pages) {
                if (lane < per_block && key < u.un_hi && key + a.box > u.un_lo) flag_status(a.status, kDevBadIndex);
                page = -1;
            }
            const unsigned there = __ballot_sync(0xFFFFFFFFu, page >= 0);
            const int row_in = kvh * a.page_size + key % a.page_size;
            for (int w = 0; w < 2; ++w, ++loads) {
                const int stage = loads % kS;
                if (!wait_on(&empty[stage], ((loads / kS) & 1) ^ 1, a, s.abort)) {
                    ok = false;
                    break;
                }
                uint8_t *dst = kCopy ? s.raw + stage * kRawBytes<kDim, kType> : kv + stage * kTileBytes<kDim>;
                if (there != (1u << per_block) - 1) {
                    for (int p = 0; p < per_block; ++p)
                        if (!(there >> p & 1)) {
                            if constexpr (kCopy) {
                                for (int i = lane; i < a.box * kR / 16; i += 32)
                                    reinterpret_cast<uint4 *>(dst + p * a.box * kR)[i] = make_uint4(0, 0, 0, 0);
                                for (int i = lane; i < a.box * kSc / 16; i += 32)
                                    reinterpret_cast<uint4 *>(dst + kBlock * kR + p * a.box * kSc)[i] = make_uint4(0, 0, 0, 0);
                            } else {
                                for (int i = lane; i < a.box * (kDim / 8); i += 32)
                                    *reinterpret_cast<uint4 *>(dst + tile_at(p * a.box + i / (kDim / 8), i % (kDim / 8))) = make_uint4(0, 0, 0, 0);
                            }
                        }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], __popc(there) * a.box * (kR + kSc));
                __syncwarp();
                if (page >= 0) {
                    if constexpr (kCopy) {
                        const int64_t row = static_cast<int64_t>(page) * a.kv_heads * a.page_size + row_in;
                        if (in_bounds(row + a.box <= a.n_pages * a.kv_heads * a.page_size, a.status)) {
                            bulk_load(dst + lane * a.box * kR, (w ? a.cv : a.ck) + row * kR, a.box * kR, &full[stage]);
                            bulk_load(dst + kBlock * kR + lane * a.box * kSc, (w ? a.cv_scale : a.ck_scale) + row * kSc, a.box * kSc, &full[stage]);
                        }
                    } else {
                        for (int c = 0; c < kDim / 64; ++c)
                            tma_load_3d(smem_u32(dst) + c * (kBlock * 128) + lane * a.box * 128, w ? map_v : map_k, &full[stage], c * 64, row_in, page);
                    }
                }
                __syncwarp();
            }
        }
    }
    // copies in flight have to land before the CTA ends, also when another role gave up
    for (int l = loads > kS ? loads - kS : 0; l < loads; ++l) mbar_wait(&full[l % kS], (l / kS) & 1, kDrainLimitNs, nullptr);
    for (int i = 0; i < 2; ++i)
        if (q_n[i] > 0) mbar_wait(&s.q_full[i], (q_n[i] - 1) & 1, kDrainLimitNs, nullptr);
}

// Warp 11: V of blocks that some row sees in part.
template <int kDim>
__device__ __forceinline__ void look_at_values(const PromptArgs &a, const Smem &s, uint8_t *kv) {
    constexpr int kS = kStages<kDim, BD_KV_BF16>;
    const int lane = threadIdx.x % 32;
    int it = 0, loads = 0;
    while (true) {
        const Unit u = next_unit(a, s, it);
        if (u.blocks < 0) return;
        for (int l = 0; l < 2 * u.blocks; ++l, ++loads) {
            const int stage = loads % kS, blk = u.blk0 + l / 2;
            if (!wait_on(&s.full[stage], (loads / kS) & 1, a, s.abort)) return;
            if (l % 2 && seen_in_part(u, blk)) {
                uint8_t *tile = kv + stage * kTileBytes<kDim>;
                bool bad = false;
                // 0 times a number is added up: not 0 where one of them is not finite
                uint32_t sum[4] = {0, 0, 0, 0};
                const int from = max(0, u.un_lo - blk * kBlock), to = min(kBlock, u.un_hi - blk * kBlock);
                if (from > 0 || to < kBlock) {
                    for (int i = lane; i < kBlock * (kDim / 8); i += 32)
                        if (i / (kDim / 8) < from || i / (kDim / 8) >= to)
                            *reinterpret_cast<uint4 *>(tile + tile_at(i / (kDim / 8), i % (kDim / 8))) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
#pragma unroll 16
                for (int i = lane; i < kBlock * (kDim / 8); i += 32) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(tile + i * 16);
                    sum[0] = zero_times(x.x, sum[0]), sum[1] = zero_times(x.y, sum[1]);
                    sum[2] = zero_times(x.z, sum[2]), sum[3] = zero_times(x.w, sum[3]);
                }
                bad = __any_sync(0xFFFFFFFFu, ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7FFF7FFFu) != 0);
                if (bad && lane == 0) s.slow[stage] = loads + 1;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.fixed[stage]);
                mbar_arrive(&s.empty[stage]);
            }
        }
    }
}

// Warps 11 to 15: tiles as they are in the cache to the bf16 numbers that they stand for, or fp16 ones of an eighth of that, 16 bytes
// at a time.
__device__ __forceinline__ uint32_t bf16_pair(__half2_raw h, uint32_t scale) {  // times a scale given twice: exact in bf16
    const float2 f = __half22float2(__half2(h));
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(pack_bf16x2(f.x, f.y)), "r"(scale));
    return r;
}
template <int kDim, int kType>
__device__ __forceinline__ void convert_tiles(const PromptArgs &a, const Smem &s, uint8_t *kv) {
    constexpr int kS = kStages<kDim, kType>, kRaw = kRawSlots<kDim, kType>, kSc = kScale<kDim, kType>;
    constexpr int kPer = kRow<kDim, kType> / 16;       // 16-byte pieces of a key
    constexpr int kOut = kType == BD_KV_E4M3 ? 2 : 4;  // and of 16-bit numbers that each makes
    constexpr int kThreads = kConvertWarps * 32, kEach = (kBlock * kPer + kThreads - 1) / kThreads;
    constexpr int kStep = kThreads / kPer;             // from a thread's key to its next
    static_assert(kThreads % kPer == 0 && kStep % 4 == 0);
    const int lane = threadIdx.x % 32, tid = threadIdx.x - 11 * 32, key_first = tid / kPer;
    // The swizzle turns with the key: by nothing from one to the next, or by 4 pieces there and back
    uint32_t at[kOut];
#pragma unroll
    for (int o = 0; o < kOut; ++o) at[o] = tile_at(key_first, tid % kPer * kOut + o);
    int it = 0, loads = 0;
    while (true) {
        const Unit u = next_unit(a, s, it);
        if (u.blocks < 0) return;
        for (int l = 0; l < 2 * u.blocks; ++l, ++loads) {
            const int stage = loads % kS, slot = loads % kRaw, key0 = (u.blk0 + l / 2) * kBlock;
            if (!wait_on(&s.raw_full[slot], (loads / kRaw) & 1, a, s.abort)) return;
            uint8_t *tile = kv + stage * kTileBytes<kDim>;
            const uint8_t *raw = s.raw + slot * kRawBytes<kDim, kType>, *scales = raw + kBlock * kRow<kDim, kType>;
            uint4 in[kEach];
            uint32_t sc[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                in[e] = make_uint4(0, 0, 0, 0), sc[e] = 0;
                if (key_first + e * kStep >= kBlock) continue;
                in[e] = reinterpret_cast<const uint4 *>(raw)[tid + e * kThreads];
                if constexpr (kType == BD_KV_E4M3) sc[e] = scales[key_first + e * kStep];
                else sc[e] = *reinterpret_cast<const uint16_t *>(scales + (key_first + e * kStep) * kSc + tid % kPer * 2);
            }
            bool bad = false;
            if (l % 2 && seen_in_part(u, u.blk0 + l / 2)) {  // rows that nobody sees are zeros; is another one not finite?
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int key = key0 + key_first + e * kStep;
                    if (key < u.un_lo || key >= u.un_hi) in[e] = make_uint4(0, 0, 0, 0), sc[e] = 0;
                    if constexpr (kType == BD_KV_E4M3) {  // a NaN byte, or a scale that may take a number past bf16's largest
                        auto nan = [](uint32_t x) { return (((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; };
                        bad |= nan(in[e].x) || nan(in[e].y) || nan(in[e].z) || nan(in[e].w) || sc[e] >= 246;
                    } else {  // scales alone can be
                        bad |= (sc[e] & 0xFFu) >= 0xF8u || sc[e] >> 8 >= 0xF8u;
                    }
                }
            }
            if (!wait_on(&s.empty[stage], ((loads / kS) & 1) ^ 1, a, s.abort)) return;
            if (bad) s.slow[stage] = loads + 1;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (key_first + e * kStep >= kBlock) continue;
                const uint32_t x[4] = {in[e].x, in[e].y, in[e].z, in[e].w};
                uint32_t scale[2];  // as a bf16 or fp16 number, twice
                if constexpr (kType == BD_KV_E4M3) {
                    scale[0] = scale[1] = sc[e] << 7 | sc[e] << 23;
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t b = (sc[e] >> 8 * h & 0xFFu) << 7;
                        scale[h] = half2_times(b | b << 16, 0x30003000u);  // an eighth: exact, to 2^-20 of its subnormals
                    }
                }
#pragma unroll
                for (int o = 0; o < kOut; ++o) {
                    uint32_t y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (kType == BD_KV_E4M3)
                            y[k] = bf16_pair(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x[2 * o + k / 2] >> k % 2 * 16 & 0xFFFFu), __NV_E4M3), scale[0]);
                        else
                            y[k] = half2_times(e2m1_pair(x[o] >> k * 8), scale[o / 2]);
                    }
                    *reinterpret_cast<uint4 *>(tile + (at[o] ^ (kStep % 8 ? e % 2 * 64 : 0)) + e * kStep * 128) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.full[stage]);
                mbar_arrive(&s.raw_empty[slot]);
            }
        }
    }
}

// ---- warps 0 to 7: softmax ----------------------------------------------------------------

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&o)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]), "=r"(o[8]), "=r"(o[9]),
          "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
        : "r"(taddr));
}

// Waits for the loads so far; what is read of v comes after.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
          "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
          "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
          "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
          "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
        :
        : "memory");
}

// cap tanh of two products given as y = 2 log2(e) / cap times their scores.  Small ones by the tangent's series (from |y| = kSmall on
// the next term passes 2^-23 of the value), whose error is relative to the score, not to cap.
constexpr float kSmall = 0.9f;  // scores of 0.31 cap
__device__ __forceinline__ float2 capped_small(float2 y, float cap) {
    const float2 x = mul2(y, make_float2(0.34657359027997f, 0.34657359027997f)), z = mul2(x, x);  // ln(2) / 2
    float2 p = fma2(z, make_float2(62.f / 2835, 62.f / 2835), make_float2(-17.f / 315, -17.f / 315));
    p = fma2(z, p, make_float2(2.f / 15, 2.f / 15));
    p = fma2(z, p, make_float2(-1.f / 3, -1.f / 3));
    return mul2(fma2(mul2(x, z), p, x), make_float2(cap, cap));
}
// Any: with e = exp(-2 |x|), tanh |x| = 2 / (1 + e) - 1.  The reciprocal is
// Newton's, two steps from (98 - 80 e + 32 e^2) / 99, which is within 1/99 for e in [0, 1]: the transcendental unit, with an
// exponential here and one for the weight, is the busier one.
__device__ __forceinline__ float2 capped(float2 y, float cap) {
    const float2 e = make_float2(ex2(-fabsf(y.x)), ex2(-fabsf(y.y)));
    const float2 one = make_float2(1.f, 1.f), minus = make_float2(-1.f, -1.f);
    const float2 q = fma2(e, minus, minus);  // -(1 + e)
    float2 r = fma2(e, fma2(e, make_float2(32.f / 99, 32.f / 99), make_float2(-80.f / 99, -80.f / 99)), make_float2(98.f / 99, 98.f / 99));
    r = fma2(r, fma2(q, r, one), r);
    r = fma2(r, fma2(q, r, one), r);
    r = fma2(r, make_float2(2.f * cap, 2.f * cap), make_float2(-cap, -cap));
    const float2 small = capped_small(y, cap);
    return make_float2(fabsf(y.x) < kSmall ? small.x : copysignf(r.x, y.x), fabsf(y.y) < kSmall ? small.y : copysignf(r.y, y.y));
}

// A row's products to capped scores, in place.  `in`: 2 log2(e) / cap of a product's score.  Apart: beside the rest of a softmax thread's loop
// its code and registers slow down calls without a cap too.
__device__ __noinline__ void cap_scores(uint32_t t_s, float in, float cap) {
#pragma unroll 1
    for (int c = 0; c < kBlock; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(t_s + c, v);
        tmem_ld_wait_for(v);
        float largest = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 y = mul2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), make_float2(in, in));
            largest = max3(largest, fabsf(y.x), fabsf(y.y));
            v[i] = __float_as_uint(y.x), v[i + 1] = __float_as_uint(y.y);
        }
        auto each = [&](auto cap_of) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 y = cap_of(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                v[i] = __float_as_uint(y.x), v[i + 1] = __float_as_uint(y.y);
            }
        };
        if (__any_sync(0xFFFFFFFFu, largest >= kSmall)) each([&](float2 y) { return capped(y, cap); });
        else each([&](float2 y) { return capped_small(y, cap); });
        tmem_st_32x32b_x32(t_s + c, v);
    }
    tmem_st_wait();
}

// The rows' output so far, times f.  Seldom run: apart, so that its registers are not the loop's.
template <int kDim>
__device__ __noinline__ void scale_output(uint32_t t_o, float f) {
#pragma unroll 1
    for (int c = 0; c < kDim; c += 16) {
        uint32_t o[16];
        tmem_ld_x16(t_o + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st_32x32b_x16(t_o + c, o);
    }
    tmem_st_wait();
}

// P V of a block whose V is not finite where some row does not see it: row by row over the keys [from, to) that the row
// sees, whose weights are read from tensor memory in pairs, first and second parts.
template <int kDim, bool half>
__device__ __noinline__ void add_values(uint32_t t_p, uint32_t t_o, const uint8_t *v, bool fresh, int from, int to, unsigned missing) {
#pragma unroll 1
    for (int c = 0; c < kDim; c += 16) {
        uint32_t o[16] = {};
        if (!fresh) tmem_ld_x16(t_o + c, o);
        tmem_ld_wait();
#pragma unroll 1
        for (int k = 0; k < kBlock; ++k) {
            const float2 one = unpack_pair<half>(__float_as_uint(tmem_ld_one(t_p + weight_at(k))));
            const float2 two = unpack_pair<half>(__float_as_uint(tmem_ld_one(t_p + weight_at(k) + 8)));
            if (k >= from && k < to && !(missing >> k / 16 & 1)) {
                const float w = k % 2 ? one.y + two.y : one.x + two.x;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(v + tile_at(k, c / 8 + h));
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack_pair<half>(in[i]);
                        o[8 * h + 2 * i] = __float_as_uint(fmaf(w, f.x, __uint_as_float(o[8 * h + 2 * i])));
                        o[8 * h + 2 * i + 1] = __float_as_uint(fmaf(w, f.y, __uint_as_float(o[8 * h + 2 * i + 1])));
                    }
                }
            }
            __syncwarp();
        }
        tmem_st_32x32b_x16(t_o + c, o);
    }
    tmem_st_wait();
}

__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1; }

// Which of a block's 8 pieces of 16 keys have a page id out of range.
__device__ __noinline__ unsigned missing_pieces(const PromptArgs &a, const Unit &u, int blk) {
    const int lane = threadIdx.x % 32, key = blk * kBlock + lane * 16;
    bool fine = true;
    if (lane < 8 && key < u.un_hi && key + 16 > u.un_lo) {
        const int at = key / a.page_size;
        fine = false;
        if (in_bounds(at >= 0 && at < a.max_pages, a.status)) {
            const int32_t page = a.page_table[static_cast<int64_t>(u.seq) * a.max_pages + at];
            fine = page >= 0 && page < a.n_pages;
        }
    }
    return ~__ballot_sync(0xFFFFFFFFu, fine) & 0xFFu;
}

// A row of Q in shared memory to fp16, times the power of two that brings its largest value to [2^14, 2^15), so that values down to
// 2^-31 of it are as they were; what the products have to be multiplied by (NaN for a row that is not finite).  2^127 is the largest
// such power: times that, bf16's smallest number is 2^-6 and a row of small numbers is as it was.
template <int kDim>
__device__ __forceinline__ float query_to_half(uint8_t *q, int r) {
    uint32_t top2 = 0;
#pragma unroll 4
    for (int c = 0; c < kDim / 8; ++c) {
        const uint4 x = *reinterpret_cast<const uint4 *>(q + tile_at(r, c));
        top2 = __vmaxu2(__vmaxu2(top2, x.x & 0x7FFF7FFFu), __vmaxu2(x.y & 0x7FFF7FFFu, __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
    }
    const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    const int e = max(14, min(254, static_cast<int>(top >> 7)));
    const float up = __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);
#pragma unroll 4
    for (int c = 0; c < kDim / 8; ++c) {
        uint4 *p = reinterpret_cast<uint4 *>(q + tile_at(r, c));
        const uint4 x = *p;
        auto turn = [&](uint32_t v) { return pack_half2(bf16lo_to_f32(v) * up, bf16hi_to_f32(v) * up); };
        *p = make_uint4(turn(x.x), turn(x.y), turn(x.z), turn(x.w));
    }
    return top >= 0x7F80u ? NAN : __uint_as_float(static_cast<uint32_t>(e - 14 + 3) << 23);  // keys enter as an eighth
}

template <int kDim, int kType>
__device__ __forceinline__ void softmax_rows(const PromptArgs &a, const Smem &s, uint32_t tmem, const uint8_t *kv) {
    constexpr int kS = kStages<kDim, kType>;
    const int tile = threadIdx.x / 128, r = threadIdx.x % 128, lane = threadIdx.x % 32;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(r / 32 * 32) << 16);
    const uint32_t t_s = lane_base + tile * kBlock, t_o = lane_base + 2 * kBlock + tile * kDim;
    int s_n = 0, blocks_before = 0;
    [[maybe_unused]] uint32_t q_round = 0;
    for (int it = 0;; ++it) {
        if (!wait_on(&s.u_full[it & 1], (it >> 1) & 1, a, s.abort)) return;
        const Unit &u = s.unit[it & 1];  // held until its rows are written
        const int blocks = u.blocks;
        if (blocks < 0) return;
        const bool mine = tile == 0 || u.tokens > a.tile_tokens;
        if (mine) {
            // this thread's row
            const int token = r / a.heads_tile, t = tile * a.tile_tokens + token;
            const int head_in = u.vh % a.subs * a.heads_tile + r - token * a.heads_tile, head = u.vh / a.subs * a.group + head_in;
            const int64_t row = static_cast<int64_t>(u.row0) + t;
            const int p = u.pos0 + t;
            const bool write = token < a.tile_tokens && t < u.tokens && head_in < a.group &&
                               in_bounds(row >= 0 && row < a.total && head < a.q_heads, a.status);
            int lo = 0, hi = INT_MAX;  // rows without a query see everything, to no effect
            float slope = 0.f;
            bool none = false;
            if (write) {
                hi = max(p + 1, u.prefix);
                lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
                if (a.first) lo = max(lo, a.first[row]);
                none = p < 0 || lo >= hi;
                if (none) lo = 0, hi = INT_MAX;
                if (a.slopes) slope = a.slopes[head] * 1.44269504088896f;
            }
            const int key_first = u.blk0 * kBlock, in_lo = u.in_lo, in_hi = u.in_hi;
            const bool gaps = u.state & kGaps;
            float unit = a.scale_log2;  // of a product
            if constexpr (kHalf<kType>)
                if (blocks > 0) {
                    if (!wait_on(&s.q_full[tile], q_round, a, s.abort)) return;
                    q_round ^= 1;
                    unit *= query_to_half<kDim>(const_cast<uint8_t *>(kv) - (2 - tile) * kTileBytes<kDim>, r);
                    // plain scores are multiplied by it after the masks: it may not be 0.  Products are below 2^36, so these scores are 0
                    if (a.plain && unit < 0x1p-126f) unit = 0x1p-126f;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.q_ready[tile]);
                }
            float top = -INFINITY, sum = 0.f;
            for (int j = 0; j < blocks; ++j) {
                const int key0 = key_first + j * kBlock;
                if (!wait_on(&s.s_full[tile], s_n & 1, a, s.abort)) return;
                tc_fence_after();
                const int from = lo - key0, to = hi - key0;
                unsigned missing = 0;
                if (gaps) missing = missing_pieces(a, u, key0 / kBlock);
                const bool part = key0 < in_lo || key0 + kBlock > in_hi;  // some row sees the block in part
                if (a.cap > 0.f) cap_scores(t_s, unit * a.cap_in, a.cap);
                const bool rewrite = !(a.plain || a.cap > 0.f) || a.slopes || part || missing;
                const float far = static_cast<float>(p - key0);
                auto rule = [&](uint32_t(&v)[32], int c) {  // on the scores of keys c ..
                    if (!a.plain && !(a.cap > 0.f)) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y = mul2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), make_float2(unit, unit));
                            v[i] = __float_as_uint(y.x), v[i + 1] = __float_as_uint(y.y);
                        }
                    }
                    if (a.slopes) {
                        const float first = far - static_cast<float>(c);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(fmaf(-slope, fabsf(first - static_cast<float>(i)), __uint_as_float(v[i])));
                    }
                    if (part || missing) {  // a bit for each key
                        const unsigned two = missing >> c / 16;
                        const uint32_t gone = (two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u);
                        const uint32_t seen = bits_below(to - c) & ~bits_below(from - c) & ~gone;
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = seen >> i & 1 ? v[i] : 0xFF800000u;  // -infinity
                    }
                    tmem_st_32x32b_x32(t_s + c, v);
                };
                // Caps, biases and masks are applied in place in tensor memory, 32 keys at a time, and the scores are read twice, 32 at a
                // time with the next under way: a row held in registers and its code unrolled are more than the registers and the
                // instruction caches have room for (8192 tokens, bf16: 486 us, 526 held).
                uint32_t x[2][32];
                float most[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) most[c] = -INFINITY;  // chains short enough to hide an operation's latency
                auto look = [&](const uint32_t(&v)[32], float *m) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) m[k] = max3(m[k], __uint_as_float(v[i + k]), __uint_as_float(v[i + k + 4]));
                };
                tmem_ld_32x32b_x32(t_s, x[0]);
#pragma unroll 1
                for (int c = 0; c < kBlock; c += 64) {
                    tmem_ld_wait_for(x[0]);
                    tmem_ld_32x32b_x32(t_s + c + 32, x[1]);
                    if (rewrite) rule(x[0], c);
                    look(x[0], most);
                    tmem_ld_wait_for(x[1]);
                    if (rewrite) tmem_st_wait();
                    tmem_ld_32x32b_x32(t_s + (c + 64) % kBlock, x[0]);  // the next, or the first again
                    if (rewrite) rule(x[1], c + 32);
                    look(x[1], most + 4);
                }
                if (rewrite) tmem_st_wait();
                const float scale = a.plain ? unit : 1.f;
                const float now = fmaxf(max3(max3(most[0], most[1], most[2]), most[3], most[4]), max3(most[5], most[6], most[7])) * scale;
                const bool raise = now > top + kLazy<kType> || (top == -INFINITY && now > top);
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    float fix = 1.f;
                    if (raise) {
                        if (top != -INFINITY) fix = ex2(top - now), sum *= fix;
                        top = now;
                    }
                    if (__any_sync(0xFFFFFFFFu, fix != 1.f)) {  // not in the first block, where nothing was held yet
                        if (!wait_on(&s.o_full[tile], (s_n - 1) & 1, a, s.abort)) return;
                        tc_fence_after();
                        tmem_ld_wait_for(x[0]);
                        scale_output<kDim>(t_o, fix);
                    }
                }
                const float base = (top == -INFINITY ? 0.f : top) - kLift<kType>;
                float2 add[2] = {};
                auto weights = [&](const uint32_t(&v)[32], int c) {  // of keys c ..
                    const float2 scale2 = make_float2(scale, scale), base2 = make_float2(-base, -base);
#pragma unroll
                    for (int k = 0; k < 32; k += 16) {
                        uint32_t w[16];  // first parts, second parts
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float2 e = fma2(make_float2(__uint_as_float(v[k + 2 * i]), __uint_as_float(v[k + 2 * i + 1])), scale2, base2);
                            e.x = ex2(e.x), e.y = ex2(e.y);
                            add[i % 2] = add2(add[i % 2], e);
                            w[i] = kHalf<kType> ? pack_half2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                            const float2 left = fma2(unpack_pair<kHalf<kType>>(w[i]), make_float2(-1.f, -1.f), e);  // exact
                            w[8 + i] = kHalf<kType> ? pack_half2(left.x, left.y) : pack_bf16x2(left.x, left.y);
                        }
                        tmem_st_32x32b_x16(t_s + c + k, w);
                    }
                };
                auto hand_over = [&](int half) {  // 64 keys: their product may begin
                    if (part) return;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.p_full[2 * tile + half]);
                };
#pragma unroll 1
                for (int c = 0; c < kBlock; c += 64) {
                    tmem_ld_wait_for(x[0]);
                    tmem_ld_32x32b_x32(t_s + c + 32, x[1]);
                    weights(x[0], c);
                    tmem_ld_wait_for(x[1]);
                    if (c == 0) tmem_ld_32x32b_x32(t_s + 64, x[0]);
                    weights(x[1], c + 32);
                    hand_over(c / 64);
                }
                if (part) {  // is V finite where it is not seen?
                    const int load = 2 * (blocks_before + j) + 1, stage = load % kS;
                    if (!wait_on(kType == BD_KV_BF16 ? &s.fixed[stage] : &s.full[stage], (load / kS) & 1, a, s.abort)) return;
                    tmem_st_wait();
                    if (s.slow[stage] == load + 1) {
                        if (j > 0 && !wait_on(&s.o_full[tile], (s_n - 1) & 1, a, s.abort)) return;
                        tc_fence_after();
                        add_values<kDim, kHalf<kType>>(t_s, t_o, kv + stage * kTileBytes<kDim>, j == 0, from, to, missing);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.p_full[2 * tile]), mbar_arrive(&s.p_full[2 * tile + 1]);
                }
                sum += (add[0].x + add[1].x) + (add[0].y + add[1].y);
                ++s_n;
            }
            // the unit's rows
            if (blocks > 0) {
                if (!wait_on(&s.o_full[tile], (s_n - 1) & 1, a, s.abort)) return;
                tc_fence_after();
            }
            const bool whole = u.slot < 0;
            float *part = nullptr;
            if (!whole && in_bounds(u.slot < a.slots, a.status)) part = a.parts + u.slot * kSlotFloats<kDim> + tile * (kTileRows * (kDim + 2));
            if (none || blocks == 0) sum = 0.f, top = -INFINITY;
            const bool empty = sum == 0.f;
            const float inv = empty ? 0.f : (kHalf<kType> ? 8.f : 1.f) / sum;
            top -= kLift<kType>;
            uint8_t *dst = a.out + (row * a.q_heads + head) * (kDim * 2);
#pragma unroll 1
            for (int c = 0; c < kDim; c += 32) {
                uint32_t o[32];
                if (blocks > 0) {
                    tmem_ld_32x32b_x32(t_o + c, o);
                    tmem_ld_wait();
                }
                if (empty)
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0;
                if (whole) {
                    if (write)
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            float f[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(o[i + k]) * inv;
                            *reinterpret_cast<uint4 *>(dst + (c + i) * 2) = pack8(f);
                        }
                } else if (part) {  // columns in fours, each of all rows side by side
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        reinterpret_cast<uint4 *>(part)[(c + i) / 4 * kTileRows + r] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
            if (whole) {
                if (write && a.lse) a.lse[row * a.q_heads + head] = empty ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
            } else if (part) {
                part[kTileRows * kDim + r] = top;
                part[kTileRows * (kDim + 1) + r] = sum;
                if (threadIdx.x == 0 && (u.state & kFirstPiece)) a.heads[u.slot] = make_int4(u.parts, u.row0, u.tokens, u.vh);
            }
            tc_fence_before();  // the reads of O come before the next unit's first product
        }
        blocks_before += blocks;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.u_empty[it & 1]);
    }
}

template <int kDim, int kType>
__global__ void __launch_bounds__(kThreadsOf<kType>, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PromptArgs a) {
    constexpr int kS = kStages<kDim, kType>;
    constexpr bool kConvert = kType != BD_KV_BF16;
    uint8_t *smem = smem_raw + (smem_base() - smem_u32(smem_raw));
    uint8_t *kv = smem + 2 * kTileBytes<kDim>;
    Smem s;
    s.raw = kv + kS * kTileBytes<kDim>;
    uint64_t *bars = reinterpret_cast<uint64_t *>(s.raw + kRawSlots<kDim, kType> * kRawBytes<kDim, kType>);
    s.full = bars, s.empty = bars + kS, s.fixed = bars + 2 * kS;
    bars += 3 * kS;
    s.raw_full = bars, s.raw_empty = bars + 4;
    bars += 8;
    s.q_full = bars, s.q_empty = bars + 2, s.s_full = bars + 4, s.o_full = bars + 6;  // o_full[2]: the last products
    s.p_full = bars + 9;                                                            // of each tile: the first and second 64 keys
    s.u_full = bars + 13, s.u_empty = bars + 15;
    s.q_ready = bars + 17;
    s.u_want = bars + 19;
    s.unit = reinterpret_cast<Unit *>(bars + 20);
    s.slow = reinterpret_cast<volatile int *>(s.unit + 2);
    s.abort = s.slow + kS;
    s.tmem = const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(s.abort + 1));
    static_assert(kRawSlots<kDim, kType> <= 4 && (3 * kS + 28) * 8 + 2 * sizeof(Unit) + (kS + 2) * 4 <= 1024);
    const int warp = threadIdx.x / 32;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            mbar_init(&s.full[i], kConvert ? kConvertWarps : 1);
            mbar_init(&s.empty[i], kConvert ? 1 : 2);  // the products that read it, and warp 11
            mbar_init(&s.fixed[i], 1);
            s.slow[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1), mbar_init(&s.q_ready[i], 4), mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1), mbar_init(&s.o_full[i], 1);
            mbar_init(&s.p_full[2 * i], 4), mbar_init(&s.p_full[2 * i + 1], 4);
            mbar_init(&s.u_full[i], 1), mbar_init(&s.u_empty[i], 10 + (kConvert ? kConvertWarps : 1));
        }
        for (int i = 0; i < kRawSlots<kDim, kType>; ++i) mbar_init(&s.raw_full[i], 1), mbar_init(&s.raw_empty[i], kConvertWarps);
        mbar_init(&s.o_full[2], 1);
        mbar_init(s.u_want, 1);
        *s.abort = 0;
        mbar_fence_init();
        tma_prefetch_desc(&map_q);
        if (!kConvert) tma_prefetch_desc(&map_k), tma_prefetch_desc(&map_v);
    }
    if (warp == 8) {
        tmem_alloc(s.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    pdl_wait();  // what came before on the stream is complete; the set-up above needed nothing of it
    // where units are split, CTA b takes unit b alone: its slot holds no unit's first piece yet
    if (threadIdx.x == 0 && a.may_split && in_bounds(static_cast<int>(blockIdx.x) < a.slots, a.status)) a.heads[blockIdx.x] = make_int4(0, 0, 0, 0);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s.tmem;  // 0: all of it is this CTA's
    // softmax threads hold most: 384 threads start with 168 registers each, 512 with 128
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConvert ? 184 : 216));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp < 8) {
        softmax_rows<kDim, kType>(a, s, 0, kv);
    } else if (warp == 8) {
        if (elect_one()) issue_products<kDim, kType>(a, s);
        __syncwarp();
    } else if (warp == 9) {
        find_units(a, s);
    } else if (warp == 10) {
        load_tiles<kDim, kType>(a, s, &map_q, &map_k, &map_v, smem_base(), kv);
    } else if constexpr (kConvert) {
        convert_tiles<kDim, kType>(a, s, kv);
    } else {
        look_at_values<kDim>(a, s, kv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// ---- join of the pieces ---------------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;

// A CTA per slot, tile and 32 rows; a thread has a row and an eighth of its columns.  Pieces of a unit are vheads slots apart.
template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const __grid_constant__ PromptArgs a) {
    pdl_trigger_and_wait();
    const int4 h = a.heads[blockIdx.x];
    const int pieces = h.x, tile = blockIdx.y / (kTileRows / kJoinRows);
    if (pieces < 1) return;
    const int r = blockIdx.y % (kTileRows / kJoinRows) * kJoinRows + threadIdx.x % kJoinRows, eighth = threadIdx.x / kJoinRows;
    const int vheads = a.kv_heads * a.subs;
    const int token = r / a.heads_tile, t = tile * a.tile_tokens + token, head_in = h.w % a.subs * a.heads_tile + r - token * a.heads_tile;
    if (token >= a.tile_tokens || t >= h.z || head_in >= a.group) return;
    const int64_t row = static_cast<int64_t>(h.y) + t;
    const int head = h.w / a.subs * a.group + head_in;
    if (!in_bounds(row < a.total && head < a.q_heads && blockIdx.x + (pieces - 1) * vheads < a.slots, a.status)) return;
    auto part = [&](int q) { return a.parts + (blockIdx.x + static_cast<int64_t>(q) * vheads) * kSlotFloats<kDim> + tile * (kTileRows * (kDim + 2)); };
    float top = -INFINITY;
    for (int q = 0; q < pieces; ++q) top = fmaxf(top, part(q)[kTileRows * kDim + r]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float4 o[kDim / 32] = {};
    for (int q = 0; q < pieces; ++q) {
        const float *p = part(q);
        const float f = ex2(p[kTileRows * kDim + r] - base);
        sum = fmaf(p[kTileRows * (kDim + 1) + r], f, sum);
#pragma unroll
        for (int i = 0; i < kDim / 32; ++i) {
            const float4 y = reinterpret_cast<const float4 *>(p)[(eighth * (kDim / 32) + i) * kTileRows + r];
            o[i].x = fmaf(y.x, f, o[i].x), o[i].y = fmaf(y.y, f, o[i].y), o[i].z = fmaf(y.z, f, o[i].z), o[i].w = fmaf(y.w, f, o[i].w);
        }
    }
    const float inv = sum == 0.f ? 0.f : a.v_unit / sum;
    uint2 *dst = reinterpret_cast<uint2 *>(a.out + (row * a.q_heads + head) * (kDim * 2)) + eighth * (kDim / 32);
#pragma unroll
    for (int i = 0; i < kDim / 32; ++i)
        dst[i] = make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
    if (a.lse && eighth == 0) a.lse[row * a.q_heads + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
}

size_t table_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * sizeof(int4) + 255) / 256 * 256; }
template <int kDim>
size_t part_bytes(int num_sms) { return static_cast<size_t>(num_sms) * kSlotFloats<kDim> * 4; }

template <class... Types, class... Args>
cudaError_t launch_pdl(void (*kernel)(Types...), dim3 grid, int threads, int smem, cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int kDim, int kType>
cudaError_t launch_typed(const PromptArgs &a, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const DevCtx &ctx,
                         cudaStream_t stream) {
    cudaError_t e = allow_smem<prompt_kernel<kDim, kType>>(kSmemBytes<kDim, kType>, ctx.device);
    if (e != cudaSuccess) return e;
    e = launch_pdl(prompt_kernel<kDim, kType>, dim3(ctx.num_sms), kThreadsOf<kType>, kSmemBytes<kDim, kType>, stream, q, k, v, a);
    if (e != cudaSuccess || !a.may_split) return e;
    return launch_pdl(prompt_join_kernel<kDim>, dim3(a.slots, 2 * kTileRows / kJoinRows), kJoinThreads, 0, stream, a);
}

template <int kDim>
cudaError_t launch_dim(const PromptArgs &a, int type, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const DevCtx &ctx,
                       cudaStream_t stream) {
    if (type == BD_KV_E4M3) return launch_typed<kDim, BD_KV_E4M3>(a, q, k, v, ctx, stream);
    if (type == BD_KV_E2M1) return launch_typed<kDim, BD_KV_E2M1>(a, q, k, v, ctx, stream);
    return launch_typed<kDim, BD_KV_BF16>(a, q, k, v, ctx, stream);
}

}  // namespace

// Behind what single tokens' attention uses, so that one workspace does for both.  The counts come first, so that they are where
// every call looks for them, whatever its head_dim.
size_t prompt_workspace_size(int num_sms, int head_dim) {
    return attention_workspace_size(num_sms) + 256 + table_bytes(num_sms) + (head_dim == 128 ? part_bytes<128>(num_sms) : part_bytes<64>(num_sms));
}

cudaError_t launch_prompt(const bd_kv_cache &c, const void *q, int32_t q_heads, const int32_t *offsets, int64_t total,
                          const int32_t *page_table, const int32_t *lengths, int32_t n_seqs, int32_t max_pages,
                          const bd_score_rule &rule, void *out, float *lse, void *workspace, const DevCtx &ctx,
                          cudaStream_t stream) {
    constexpr float kLog2e = 1.44269504088896f;
    PromptArgs a = {};
    a.ck = static_cast<const uint8_t *>(c.k);
    a.cv = static_cast<const uint8_t *>(c.v);
    a.ck_scale = c.k_scale;
    a.cv_scale = c.v_scale;
    a.page_table = page_table;
    a.offsets = offsets;
    a.lengths = lengths;
    a.first = rule.first;
    a.prefix = rule.prefix;
    a.slopes = rule.slopes;
    a.out = static_cast<uint8_t *>(out);
    a.lse = lse;
    uint8_t *ws = static_cast<uint8_t *>(workspace) + attention_workspace_size(ctx.num_sms);
    a.taken = reinterpret_cast<unsigned *>(ws);
    a.heads = reinterpret_cast<int4 *>(ws + 256);
    a.parts = reinterpret_cast<float *>(ws + 256 + table_bytes(ctx.num_sms));
    a.status = ctx.status;
    a.wait_ns = ctx.wait_ns;
    a.n_pages = c.n_pages;
    a.total = total;
    a.n_seqs = n_seqs;
    a.max_pages = max_pages;
    a.page_size = c.page_size;
    a.kv_heads = c.kv_heads;
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.subs = (a.group + kTileRows - 1) / kTileRows;
    a.heads_tile = (a.group + a.subs - 1) / a.subs;
    a.tile_tokens = kTileRows / a.heads_tile;
    a.window = rule.window;
    a.slots = ctx.num_sms;
    a.box = 16;
    while (a.box < kBlock && c.page_size % (2 * a.box) == 0) a.box *= 2;
    a.scale_log2 = rule.scale * kLog2e;
    a.cap = rule.cap * kLog2e;
    a.cap_in = rule.cap > 0.f ? 2.f / rule.cap : 0.f;
    a.v_unit = c.kv_type == BD_KV_E2M1 ? 8.f : 1.f;
    a.plain = rule.scale > 0.f && !(rule.cap > 0.f) && !rule.slopes;
    // The units are at least this many (offsets[n_seqs] = total): more than CTAs are not split.  Sequences of less than a unit's tokens make
    // more, a unit each: past the number of CTAs the time steps up to whole sequences' keys in turn (4 tokens or fewer of each over up to
    // 30000, 8 KV heads, bf16: 16 sequences 129 us, 18 214, 20 446, 64 477)
    const int64_t units = (total + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens) * c.kv_heads * a.subs;
    a.may_split = units <= ctx.num_sms && max_pages * static_cast<int64_t>(c.page_size) > 4 * kBlock;
    CUtensorMap map_q, map_k, map_v;
    if (!encode_tensor_map_3d(&map_q, q, c.head_dim, q_heads, total, c.head_dim * 2, static_cast<uint64_t>(q_heads) * c.head_dim * 2,
                              64, a.heads_tile, a.tile_tokens))
        return cudaErrorInvalidValue;
    map_k = map_v = map_q;
    if (c.kv_type == BD_KV_BF16) {
        const uint64_t rows = static_cast<uint64_t>(c.kv_heads) * c.page_size, page = rows * c.head_dim * 2;
        if (!encode_tensor_map_3d(&map_k, c.k, c.head_dim, rows, c.n_pages, c.head_dim * 2, page, 64, a.box, 1) ||
            !encode_tensor_map_3d(&map_v, c.v, c.head_dim, rows, c.n_pages, c.head_dim * 2, page, 64, a.box, 1))
            return cudaErrorInvalidValue;
    }
    return c.head_dim == 128 ? launch_dim<128>(a, c.kv_type, map_q, map_k, map_v, ctx, stream)
                             : launch_dim<64>(a, c.kv_type, map_q, map_k, map_v, ctx, stream);
}

}  // namespace bd
