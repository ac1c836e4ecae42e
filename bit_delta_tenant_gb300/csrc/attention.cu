// attention.cu -- attention of one new token per sequence over a paged
// key-value cache, split over the cache's length and joined.
//
//   o = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),  s_j = scale * q . K_j
//
// Bound: HBM (each K and V element is used by the few query heads that share
// its KV head).  One pass over the cache with a running maximum and sum.
//
// Work.  The keys of every (sequence, KV head) are cut into blocks of 64;
// the blocks of the whole batch, numbered sequence by sequence, head by head,
// are split evenly over the resident CTAs, so ragged lengths leave no CTA idle
// and the host needs no length.  A CTA streams its range; where the range ends
// inside a (sequence, head) it leaves the unnormalised output, maximum and sum
// of its part in the workspace, and the last part to arrive joins all parts in
// key order.  No CTA waits for another.
//
// A warp.  Each of the four warps owns 16 keys of a block and keeps its own
// running state; 16 keys of one page and head are one contiguous piece of
// memory, copied with cp.async into the warp's own ring (swizzled so that the
// fragment loads meet no bank conflict).  Query heads are the rows of
// m16n8k16: S = Q K^T, then O += P V with the score fragment reused as P's.
// mma.sync, not tcgen05: 4 to 16 rows of a 128-row tile would be used, and the
// kernel needs under a tenth of the legacy rate.
//
// Rounding.  P enters as a 16-bit part and its remainder.  With at most 8 query
// heads the remainder takes rows 8..15 of the same product, which would
// otherwise be empty; with more it takes a second product.
// e4m3 keys and values become fp16 (exact); q is scaled by a power of two into
// fp16's range, K's scale multiplies the score, and V's scale is folded into
// the weight before the maximum is taken, so that weights never exceed 1.
#include <cuda_fp8.h>

#include <algorithm>

#include "bd_device.cuh"
#include "bd_internal.h"

namespace bd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;              // keys of a warp's step
constexpr int kBlock = kWarps * kTile; // keys of a work item
constexpr int kRows = 16;              // query heads of one tile
constexpr int kCtasPerSm = 3;
constexpr int64_t kMaxKeys = 0x7FFFF000;  // positions stay int32, a block beyond the last one included
constexpr int kSlotFloats = kRows * 128 + 2 * kRows;  // a part's output, maxima and sums

struct AttnArgs {
    const uint8_t *q, *ck, *cv, *ck_scale, *cv_scale;
    const int32_t *page_table, *lengths;
    uint8_t *out;
    float *lse, *parts;
    int32_t *counters;
    unsigned *status;
    int64_t n_pages;
    int32_t n_seqs, max_pages, kv_heads, page_size, q_heads, group, subs, window;
    float scale_log2;  // scale * log2(e): scores are kept in base 2
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool full) {
    const int n = full ? 16 : 0;  // 0: nothing is read, 16 zero bytes are written
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
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
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    return static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// The 16-bit pair nearest to (x, y), and the pair nearest to what that leaves.
template <bool kHalf>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo) {
    if constexpr (kHalf) {
        hi = pack_half2(x, y);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        lo = pack_half2(x - f.x, y - f.y);
    } else {
        hi = pack_bf16x2(x, y);
        lo = pack_bf16x2(x - bf16lo_to_f32(hi), y - bf16hi_to_f32(hi));
    }
}

// Byte offset of 16-byte chunk c of row r in a tile of kRow-byte rows: eight rows of one
// chunk column fall into eight different 16-byte bank groups.
template <int kRow>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    if constexpr (kRow == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) * 16);
    return r * kRow + ((c ^ (r & 7)) * 16);
}

// What a sequence's query sees: keys [start, len), cut into `blocks` blocks from block `first`.
struct Span {
    int32_t start, len, first, blocks;
};
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
    return s;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (static_cast<int>(threadIdx.x % 32) >= o) v += u;
    }
    return v;
}

template <int kDim, bool kE4m3>
constexpr int tile_bytes() {
    return kTile * kDim * (kE4m3 ? 1 : 2);
}
template <int kDim, bool kE4m3>
constexpr int stage_bytes() {  // K tile, V tile, and their 16 scale bytes each
    return 2 * tile_bytes<kDim, kE4m3>() + (kE4m3 ? 32 : 0);
}
template <bool kE4m3>
constexpr int ring_depth() {
    return kE4m3 ? 4 : 2;
}
template <int kDim, bool kE4m3>
constexpr int smem_bytes() {
    return kWarps * ring_depth<kE4m3>() * stage_bytes<kDim, kE4m3>();
}

// kPack: at most 8 query heads, the remainders of P in rows 8..15.
template <int kDim, bool kE4m3, bool kPack>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attention_kernel(const AttnArgs a) {
    constexpr int kRow = kDim * (kE4m3 ? 1 : 2);  // bytes of one key
    constexpr int kChunks = kRow / 16;
    constexpr int kTileBytes = tile_bytes<kDim, kE4m3>();
    constexpr int kStage = stage_bytes<kDim, kE4m3>();
    constexpr int kDepth = ring_depth<kE4m3>();
    constexpr int kUsed = kPack ? 8 : 16;  // rows that carry heads
    constexpr int kSteps = kDim / 16;      // k steps of Q K^T
    constexpr int kCols = kDim / 8;        // n tiles of P V
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[kWarps];
    __shared__ int64_t s_found[2];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t4 = lane % 4;
    const int vheads = a.kv_heads * a.subs;
    pdl_trigger_and_wait();

    // sequences with nothing to see: zeros
    for (int64_t b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
        if (span_of(a, b).blocks > 0) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + b * a.q_heads * (kDim * 2));
        for (int i = tid; i < a.q_heads * (kDim / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int i = tid; i < a.q_heads; i += kThreads) a.lse[b * a.q_heads + i] = -INFINITY;
    }

    // all items, and this CTA's range of them
    int64_t mine = 0;
    for (int64_t b = tid; b < a.n_seqs; b += kThreads) mine += span_of(a, b).blocks;
    mine = warp_scan(mine);
    if (lane == 31) s_sum[warp] = mine;
    __syncthreads();
    const int64_t total = (s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) * vheads;
    const int64_t grid = min(static_cast<int64_t>(gridDim.x), total);
    if (blockIdx.x >= grid) return;
    const int64_t begin = total * blockIdx.x / grid, end = total * (blockIdx.x + 1) / grid;

    // the sequence that holds item `begin`, and the blocks before it
    {
        int64_t before = 0;
        for (int64_t b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
            __syncthreads();
            const int64_t n = b0 + tid < a.n_seqs ? span_of(a, b0 + tid).blocks : 0;
            const int64_t in = warp_scan(n);
            if (lane == 31) s_sum[warp] = in;
            __syncthreads();
            int64_t p = before + in - n;
            for (int w = 0; w < warp; ++w) p += s_sum[w];
            if (n > 0 && p * vheads <= begin && begin < (p + n) * vheads) s_found[0] = b0 + tid, s_found[1] = p;
            before += s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
        }
        __syncthreads();
    }
    int64_t b = s_found[0], blocks_before = s_found[1];
    Span sp = span_of(a, b);
    int vh = static_cast<int>((begin - blocks_before * vheads) / sp.blocks);
    int blk = static_cast<int>((begin - blocks_before * vheads) % sp.blocks);
    const uint32_t ring = smem_u32(smem) + warp * (kDepth * kStage);

    for (int64_t it = begin; it < end;) {
        const int n = static_cast<int>(min(end - it, static_cast<int64_t>(sp.blocks - blk)));
        const int kvh = vh / a.subs, row0 = vh % a.subs * kRows;
        const int rows = min(kRows, a.group - row0);
        const int64_t head0 = b * a.q_heads + kvh * a.group + row0;

        // Q fragments.  bf16: natural column order.  e4m3: the order in which a lane meets
        // four neighbouring bytes of K (slots 2t, 2t+1 and 2t+8, 2t+9 hold columns 4t .. 4t+3).
        uint32_t qa[kSteps][kPack ? 2 : 4];
        float rscale[2] = {a.scale_log2, a.scale_log2};
#pragma unroll
        for (int half = 0; half < (kPack ? 1 : 2); ++half) {
            const bool on = g + half * 8 < rows;
            const uint8_t *src = a.q + (head0 + g + half * 8) * (kDim * 2);
            uint32_t v[kSteps][2];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                if constexpr (kE4m3) {
                    const uint2 u = on ? *reinterpret_cast<const uint2 *>(src + k * 32 + t4 * 8) : make_uint2(0, 0);
                    v[k][0] = u.x, v[k][1] = u.y;
                } else {
                    v[k][0] = on ? *reinterpret_cast<const uint32_t *>(src + k * 32 + t4 * 4) : 0;
                    v[k][1] = on ? *reinterpret_cast<const uint32_t *>(src + k * 32 + 16 + t4 * 4) : 0;
                }
            }
            if constexpr (kE4m3) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = fmaxf(top, fmaxf(fabsf(bf16lo_to_f32(v[k][i])), fabsf(bf16hi_to_f32(v[k][i]))));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // q * 2^-e lies below 2 in magnitude; rows of zeros or infinities keep e = 0
                int e = static_cast<int>(__float_as_uint(top) >> 23);
                e = e < 27 || e > 227 ? 127 : e;
                const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                rscale[half] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        v[k][i] = pack_half2(bf16lo_to_f32(v[k][i]) * down, bf16hi_to_f32(v[k][i]) * down);
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                if constexpr (kPack) {
                    qa[k][0] = v[k][0], qa[k][1] = v[k][1];
                } else {
                    qa[k][half] = v[k][0], qa[k][2 + half] = v[k][1];
                }
            }
        }

        float o[kCols][4] = {};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        // this warp's 16 keys of block j of the segment
        auto key_of = [&](int j) { return (sp.first + blk + j) * kBlock + warp * kTile; };
        auto load = [&](int j) {
            const int key0 = key_of(j);
            if (j < n && key0 < sp.len && key0 + kTile > sp.start) {
                const uint32_t dst = ring + j % kDepth * kStage;
                int64_t page = a.page_table[b * a.max_pages + key0 / a.page_size];
                const bool good = page >= 0 && page < a.n_pages;
                if (!good) {
                    if (lane == 0) flag_status(a.status, kDevBadIndex);
                    page = 0;
                }
                const int64_t at = (page * a.kv_heads + kvh) * a.page_size + key0 % a.page_size;
#pragma unroll
                for (int i = lane; i < kTile * kChunks; i += 32) {
                    const int r = i / kChunks, c = i % kChunks;
                    const bool seen = good && key0 + r < sp.len && key0 + r >= sp.start;
                    const uint32_t d = dst + tile_at<kRow>(r, c);
                    cp_async16(d, a.ck + at * kRow + i * 16, seen);
                    cp_async16(d + kTileBytes, a.cv + at * kRow + i * 16, seen);
                }
                if constexpr (kE4m3)
                    if (lane < 2) cp_async16(dst + 2 * kTileBytes + lane * 16, (lane ? a.cv_scale : a.ck_scale) + at, good);
                if (!good) return false;
            }
            return true;
        };
        uint32_t bad = 0;  // ring slots whose page id was out of range
        for (int j = 0; j < kDepth - 1; ++j) {
            if (!load(j)) bad |= 1u << j;
            cp_commit();
        }
        for (int j = 0; j < n; ++j) {
            const int ahead = j + kDepth - 1;
            if (!load(ahead)) bad |= 1u << (ahead % kDepth);
            else bad &= ~(1u << (ahead % kDepth));
            cp_commit();
            cp_wait<kDepth - 1>();
            __syncwarp();
            const int key0 = key_of(j);
            if (key0 < sp.len && key0 + kTile > sp.start && !(bad >> (j % kDepth) & 1)) {
                const uint32_t kt = ring + j % kDepth * kStage, vt = kt + kTileBytes;
                float s[2][4] = {};
#pragma unroll
                for (int k = 0; k < kSteps; k += kE4m3 ? 2 : 1) {
                    uint32_t r[4];
                    if constexpr (kE4m3) {
                        // matrices: keys 0..7 and 8..15 of chunk k, then of chunk k + 1
                        ldsm4(r, kt + tile_at<kRow>(lane % 16, k + lane / 16));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t b0 = e4m3x2_to_half2(r[i] & 0xFFFFu), b1 = e4m3x2_to_half2(r[i] >> 16);
                            const int kk = k + i / 2;
                            if constexpr (kPack) mma16<true>(s[i % 2], qa[kk][0], 0, qa[kk][1], 0, b0, b1);
                            else mma16<true>(s[i % 2], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
                        }
                    } else {
                        // matrices: columns 0..7 and 8..15 of the step for keys 0..7, then keys 8..15
                        ldsm4(r, kt + tile_at<kRow>(lane % 8 + lane / 16 * 8, 2 * k + lane / 8 % 2));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if constexpr (kPack) mma16<false>(s[i], qa[k][0], 0, qa[k][1], 0, r[2 * i], r[2 * i + 1]);
                            else
                                mma16<false>(s[i], qa[k][0], qa[k][1], qa[k][2], qa[k][3], r[2 * i], r[2 * i + 1]);
                        }
                    }
                }
                // scores in base 2, V's scale exponent beside them, unseen keys -inf
                float lv[2][2] = {};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int key = i * 8 + t4 * 2 + c;
                        float ks = 1.f;
                        if constexpr (kE4m3) {
                            const uint8_t *sc = smem + (vt - smem_u32(smem)) + kTileBytes;
                            ks = __uint_as_float(static_cast<uint32_t>(sc[key]) << 23);
                            lv[i][c] = static_cast<float>(static_cast<int>(sc[16 + key]) - 127);
                        }
                        const bool seen = key0 + key < sp.len && key0 + key >= sp.start;
                        s[i][c] = seen ? s[i][c] * ks * rscale[0] : -INFINITY;
                        if (!kPack) s[i][2 + c] = seen ? s[i][2 + c] * ks * rscale[1] : -INFINITY;
                    }
                float fix[2] = {1.f, 1.f};
#pragma unroll
                for (int h = 0; h < (kPack ? 1 : 2); ++h) {
                    float top = fmaxf(fmaxf(s[0][2 * h] + lv[0][0], s[0][2 * h + 1] + lv[0][1]),
                                      fmaxf(s[1][2 * h] + lv[1][0], s[1][2 * h + 1] + lv[1][1]));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    top = fmaxf(top, m[h]);
                    const float base = top == -INFINITY ? 0.f : top;  // nothing yet: all weights 0
                    fix[h] = exp2f(m[h] - base);
                    m[h] = top;
                    l[h] *= fix[h];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float &x = s[i][2 * h + c];
                            const float e = exp2f(x - base);
                            l[h] += e;
                            x = kE4m3 ? exp2f(x + lv[i][c] - base) : e;
                        }
                }
                if constexpr (kPack) fix[1] = fix[0];
                if (__any_sync(0xFFFFFFFFu, fix[0] != 1.f || fix[1] != 1.f)) {
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        o[c][0] *= fix[0], o[c][1] *= fix[0];
                        o[c][2] *= fix[1], o[c][3] *= fix[1];
                    }
                }
                uint32_t p[4], p2[4];  // P and, for kPack false, its remainder
                if constexpr (kPack) {
                    split_pair<kE4m3>(s[0][0], s[0][1], p[0], p[1]);
                    split_pair<kE4m3>(s[1][0], s[1][1], p[2], p[3]);
                } else {
                    split_pair<kE4m3>(s[0][0], s[0][1], p[0], p2[0]);
                    split_pair<kE4m3>(s[0][2], s[0][3], p[1], p2[1]);
                    split_pair<kE4m3>(s[1][0], s[1][1], p[2], p2[2]);
                    split_pair<kE4m3>(s[1][2], s[1][3], p[3], p2[3]);
                }
                if constexpr (kE4m3) {
                    // rows 2t, 2t+1, 2t+8, 2t+9; the lane's piece of a row holds columns g * kCols ..,
                    // so n tile c takes columns g * kCols + c
                    constexpr int kWords = kCols / 4;
                    uint32_t w[4][kWords];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = t4 * 2 + i % 2 + i / 2 * 8;
                        const uint8_t *src = smem + (vt - smem_u32(smem));
                        if constexpr (kWords == 4) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(src + tile_at<kRow>(r, g));
                            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
                        } else {
                            const uint2 u = *reinterpret_cast<const uint2 *>(src + tile_at<kRow>(r, g / 2) + g % 2 * 8);
                            w[i][0] = u.x, w[i][1] = u.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kWords; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // bytes 2h, 2h+1 of two rows, side by side
                            const uint32_t x = __byte_perm(w[0][i], w[1][i], h ? 0x7362 : 0x5140);
                            const uint32_t y = __byte_perm(w[2][i], w[3][i], h ? 0x7362 : 0x5140);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t b0 = e4m3x2_to_half2(e ? x >> 16 : x & 0xFFFFu);
                                const uint32_t b1 = e4m3x2_to_half2(e ? y >> 16 : y & 0xFFFFu);
                                float(&d)[4] = o[4 * i + 2 * h + e];
                                mma16<true>(d, p[0], p[1], p[2], p[3], b0, b1);
                                if constexpr (!kPack) mma16<true>(d, p2[0], p2[1], p2[2], p2[3], b0, b1);
                            }
                        }
                } else {
#pragma unroll
                    for (int c = 0; c < kCols; c += 2) {
                        uint32_t r[4];
                        ldsm4_trans(r, vt + tile_at<kRow>(lane % 16, c + lane / 16));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            mma16<false>(o[c + i], p[0], p[1], p[2], p[3], r[2 * i], r[2 * i + 1]);
                            if constexpr (!kPack) mma16<false>(o[c + i], p2[0], p2[1], p2[2], p2[3], r[2 * i], r[2 * i + 1]);
                        }
                    }
                }
            }
            __syncwarp();  // the slot may be refilled
        }
        cp_wait<0>();
        __syncthreads();

        // the four warps' states, joined in shared memory
        float *merge = reinterpret_cast<float *>(smem);  // [warp][row][kDim]
#pragma unroll
        for (int h = 0; h < (kPack ? 1 : 2); ++h) {
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
            if (t4 == 0) s_m[warp][g + 8 * h] = m[h], s_l[warp][g + 8 * h] = l[h];
#pragma unroll
            for (int c = 0; c < kCols; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = kE4m3 ? (2 * t4 + e) * kCols + c : c * 8 + 2 * t4 + e;
                    merge[(warp * kUsed + g + 8 * h) * kDim + d] = kPack ? o[c][e] + o[c][2 + e] : o[c][2 * h + e];
                }
        }
        __syncthreads();
        const bool whole = blk == 0 && n == sp.blocks;
        const int64_t i0 = blocks_before * vheads + static_cast<int64_t>(vh) * sp.blocks;
        float *slot = a.parts + (2 * blockIdx.x + (it == begin ? 0 : 1)) * static_cast<int64_t>(kSlotFloats);
        for (int i = tid; i < rows * kDim; i += kThreads) {
            const int r = i / kDim, d = i % kDim;
            float top = s_m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f, acc = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(s_m[w][r] - base);
                sum += s_l[w][r] * f;
                acc += merge[(w * kUsed + r) * kDim + d] * f;
            }
            if (whole) {
                const __nv_bfloat16 y = __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);
                reinterpret_cast<__nv_bfloat16 *>(a.out)[(head0 + r) * kDim + d] = y;
                if (a.lse && d == 0) a.lse[head0 + r] = (top + log2f(sum)) * 0.693147180559945f;
            } else {
                slot[r * kDim + d] = acc;
                if (d == 0) slot[kRows * 128 + r] = top, slot[kRows * 128 + kRows + r] = sum;
            }
        }
        if (!whole) {
            const int c0 = static_cast<int>(((i0 + 1) * grid - 1) / total);
            const int c1 = static_cast<int>(((i0 + sp.blocks) * grid - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                int32_t *ctr = a.counters + b * vheads + vh;
                const int arrived = atomicAdd(ctr, 1);
                s_last = arrived == c1 - c0;
                if (s_last) *ctr = 0;  // ready for the next call
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                const int parts = c1 - c0 + 1;
                float *f = reinterpret_cast<float *>(smem);  // [part][row]: a part's factor
                auto slot_of = [&](int c) {
                    return a.parts + (2 * c + (total * c / grid >= i0 ? 0 : 1)) * static_cast<int64_t>(kSlotFloats);
                };
                for (int r = warp; r < rows; r += kWarps) {
                    float top = -INFINITY;
                    for (int c = lane; c < parts; c += 32) top = fmaxf(top, __ldcg(slot_of(c0 + c) + kRows * 128 + r));
#pragma unroll
                    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                    const float base = top == -INFINITY ? 0.f : top;
                    float sum = 0.f;
                    for (int c = lane; c < parts; c += 32) {
                        const float *sl = slot_of(c0 + c) + kRows * 128;
                        const float w = exp2f(__ldcg(sl + r) - base);
                        f[c * kRows + r] = w;
                        sum += __ldcg(sl + kRows + r) * w;
                    }
#pragma unroll
                    for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
                    if (lane == 0) {
                        s_l[0][r] = sum;
                        if (a.lse) a.lse[head0 + r] = (top + log2f(sum)) * 0.693147180559945f;
                    }
                }
                __syncthreads();
                for (int i = tid; i < rows * (kDim / 4); i += kThreads) {
                    const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int c = 0; c < parts; ++c) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(slot_of(c0 + c) + r * kDim + d));
                        const float w = f[c * kRows + r];
                        acc.x += x.x * w, acc.y += x.y * w, acc.z += x.z * w, acc.w += x.w * w;
                    }
                    const float sum = s_l[0][r];
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    *reinterpret_cast<uint2 *>(a.out + ((head0 + r) * kDim + d) * 2) =
                        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                }
            }
        }
        __syncthreads();  // shared memory is free again

        it += n;
        blk = 0;
        if (++vh == vheads && it < end) {
            vh = 0;
            blocks_before += sp.blocks;
            do sp = span_of(a, ++b);
            while (sp.blocks == 0);
        }
    }
}

template <int kDim, bool kE4m3, bool kPack>
cudaError_t launch_typed(const AttnArgs &a, int num_sms, cudaStream_t stream) {
    // the join keeps one factor per part and row in the same memory
    const int smem_size = std::max<int>(smem_bytes<kDim, kE4m3>(), num_sms * kCtasPerSm * kRows * sizeof(float));
    auto kernel = attention_kernel<kDim, kE4m3, kPack>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_size);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms * kCtasPerSm));
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

size_t part_bytes(int num_sms) {
    return static_cast<size_t>(2 * num_sms * kCtasPerSm) * kSlotFloats * sizeof(float);
}

int subs_of(int group) { return (group + kRows - 1) / kRows; }

}  // namespace

// The parts come first, at a size fixed by the device, so that the counters lie at the same place for every batch.
size_t attention_workspace_size(const bd_kv_cache &c, int32_t n_seqs, int32_t q_heads, int num_sms) {
    const size_t vheads = static_cast<size_t>(c.kv_heads) * subs_of(q_heads / c.kv_heads);
    return part_bytes(num_sms) + (static_cast<size_t>(n_seqs) * vheads * sizeof(int32_t) + 255) / 256 * 256;
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
    a.scale_log2 = scale * 1.44269504088896f;
    const bool e = c.kv_type == BD_KV_E4M3, pack = a.group <= 8;
    if (c.head_dim == 128) {
        if (e) return pack ? launch_typed<128, true, true>(a, ctx.num_sms, stream) : launch_typed<128, true, false>(a, ctx.num_sms, stream);
        return pack ? launch_typed<128, false, true>(a, ctx.num_sms, stream) : launch_typed<128, false, false>(a, ctx.num_sms, stream);
    }
    if (e) return pack ? launch_typed<64, true, true>(a, ctx.num_sms, stream) : launch_typed<64, true, false>(a, ctx.num_sms, stream);
    return pack ? launch_typed<64, false, true>(a, ctx.num_sms, stream) : launch_typed<64, false, false>(a, ctx.num_sms, stream);
}

}  // namespace bd
