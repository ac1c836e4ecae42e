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
//
// 4 bits.  K and V over 8 are fp16 numbers, exactly, whatever their scale: two values are converted and multiplied by their
// group's scale in two operations, and the products are of fp16 with q times a power of two of its own (values down to 2^-31 of
// its head's largest as they were) and the weights times 2^15 in two fp16 parts (2^-22 of a weight, or 2^-40 of the largest).  A lane reads
// a quarter of a key's 64 bytes for S and a sixteenth of four keys' for O, whose scale is one: a column group of 16.  Bound:
// latency and issue; the conversions and their multiplications are 128 operations of two clocks for 16 keys beside about 300
// others: 130001 tokens, 64 and 8 heads, 54.6 us (2.7 TB/s), 64 sequences of up to 8191, 32 and 8 heads, biased by distance, 34.9
// (2.0 TB/s); 49.6 and 32 with weights of one part, then with one tile in flight instead of three 50 and 36.
// A score rule (attention_scored.cu) takes two more transcendental operations for a capped score.  Plain, capped, biased, us, the same inputs over and over: 777 tokens,
// bf16, 9.3, 9.6, 10.5; 64 of up to 8191, bf16 44.4, 45.6, 45.5, 8 bits 34.0, 43.5, 41.9, 4 bits 32.1, 35.1, 33.3; 130001, bf16 88.5,
// 90.3, 90.2, 8 bits 56.3, 63.7, 61.2, 4 bits 55.6, 59.8, 56.8.
#include "attention.h"

namespace bd {
namespace {

int slots_of(int num_sms) { return 2 * num_sms * kMaxCtasPerSm; }
size_t part_bytes(int num_sms) { return static_cast<size_t>(slots_of(num_sms)) * kSlotFloats * sizeof(float); }

int subs_of(int group) { return (group + kRows - 1) / kRows; }

}  // namespace

// Slots and counters belong to CTAs, so the workspace has one size for every batch.
size_t attention_workspace_size(int num_sms) {
    return part_bytes(num_sms) + (static_cast<size_t>(kLevels) * slots_of(num_sms) * sizeof(int32_t) + 255) / 256 * 256;
}

cudaError_t launch_attention(const bd_kv_cache &c, const void *q, int32_t q_heads, const int32_t *page_table,
                             const int32_t *lengths, int32_t n_seqs, int32_t max_pages, const bd_score_rule &rule,
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
    a.window = rule.window;
    a.page_tiles = static_cast<uint32_t>(c.page_size / 16);
    // exact while piece * (page_tiles - 1) < 2^32: pieces stay below 2^26, page_tiles at most 64
    a.page_magic = static_cast<uint32_t>(((uint64_t{1} << 32) + a.page_tiles - 1) / a.page_tiles);
    constexpr float kLog2e = 1.44269504088896f;
    a.scale_log2 = rule.scale * kLog2e;
    a.slopes = rule.slopes;
    a.first = rule.first;
    a.cap = rule.cap * kLog2e;
    a.cap_in = rule.cap > 0.f ? 1.f / a.cap : 0.f;
    const bool scored = rule.cap > 0.f || rule.slopes || rule.first, pack = a.group <= 8;
    if (c.kv_type == BD_KV_E2M1) return launch_attention_four(a, scored, c.head_dim, pack, ctx, stream);
    return scored ? launch_attention_scored(a, c.kv_type, c.head_dim, pack, ctx, stream)
                  : launch_attention_plain(a, c.kv_type, c.head_dim, pack, ctx, stream);
}

}  // namespace bd
