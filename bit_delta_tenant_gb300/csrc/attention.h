// attention.h -- what attention.cu and the files that hold its kernels share.
#pragma once

#include "bd_internal.h"

namespace bd {

constexpr int kBf16 = BD_KV_BF16, kE4m3Type = BD_KV_E4M3, kE2m1 = BD_KV_E2M1;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;  // query heads of one tile
constexpr int kMaxCtasPerSm = 3;
constexpr int kDepth = 2;  // tiles in a warp's ring: one in use, one in flight (4 bits: three)
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
    const float *slopes;              // a score rule's; NULL: none
    const int32_t *first;
    float cap, cap_in;                // cap * log2(e), and 1 / that; 0: no cap
};


// Launches of a type of cache, by head_dim and whether at most 8 query heads share a KV head.
cudaError_t launch_attention_plain(const AttnArgs &a, int type, int dim, bool pack, const DevCtx &ctx, cudaStream_t stream);
cudaError_t launch_attention_scored(const AttnArgs &a, int type, int dim, bool pack, const DevCtx &ctx, cudaStream_t stream);
cudaError_t launch_attention_four(const AttnArgs &a, bool scored, int dim, bool pack, const DevCtx &ctx, cudaStream_t stream);

}  // namespace bd
