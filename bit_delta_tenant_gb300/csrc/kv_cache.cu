// kv_cache.cu -- writing new tokens into the paged key-value cache (rotary
// positions, quantisation) and reading cached tokens back as bf16.
//
// Bound: HBM for long inputs, latency for a decode step's few tokens.  Each input is
// read once and each output written once, in 16-byte pieces.  Written: a lane holds both
// halves of what is rotated together, so only a row's maximum is exchanged, by shuffles.
// Read: a CTA finds the places of its tokens once and then copies pieces in the output's order.
// Measured, heads of 128: 8 prompts of up to 4096 tokens, 64 and 8 heads, written in 8 bits in 40 us (5.4 TB/s), 64
// tokens, 32 and 8 heads, in 2.4 us; 64 sequences of 8 heads read in 8 bits in 59 us (6.1 TB/s), 1000 tokens in bf16 in 3.4 us;
// the same prompts written in 4 bits and read back 55 us (4.3 TB/s), 71 with the kernel for any layout, which reads each
// value of q and k twice.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "bd_device.cuh"
#include "bd_internal.h"
#include "bd_rows.cuh"

namespace bd {
namespace {

// A load that stays where it is written (the query may be rotated in place).
__device__ __forceinline__ uint4 ldg_plain(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// ---- append ----------------------------------------------------------------------------

constexpr int kAppendThreads = 128;  // per token: 64, 128, 256, 512 take 38, 40, 45, 65 us for long prompts, 3.2, 2.4, 2.4, 2.5 for 64 tokens
constexpr int kAppendAtOnce = 3;     // rows of a lane in flight

struct AppendArgs {
    const uint8_t *q, *k, *v;  // bf16
    uint8_t *q_out, *ck, *cv, *ck_scale, *cv_scale;
    const int32_t *seq_ids, *positions, *page_table;
    const float *rope;
    unsigned *status;
    int64_t rope_len, n_pages;
    int32_t q_heads, kv_heads, page_size, n_seqs, max_pages;
};

// Exponent byte (bias 127) of the smallest power of two s with top <= 448 s, kept within 2^-60 .. 2^120.
// 448 = 1.75 * 2^8, so a maximum of mantissa <= 1.75 and exponent e takes 2^(e - 8), a larger one 2^(e - 7).
__device__ __forceinline__ int scale_byte(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, 127 - 60), 127 + 120);
}

// Scale byte of a group in 4 bits: top / 6 to the nearest of 5 bits of exponent and 3 of mantissa.
__device__ __forceinline__ uint32_t group_scale_byte(float top) {
    const float t = __fdiv_rn(top, 6.f);
    if (t < 6.103515625e-5f) return static_cast<uint32_t>(__float2int_rn(t * 131072.f));  // below 2^-14: steps of 2^-17
    const uint32_t b = __float_as_uint(t);
    const uint32_t r = (b + 0x7FFFFu + (b >> 20 & 1u)) >> 20;  // 3 mantissa bits, ties to even
    return min(r - ((127u - 15u) << 3), 0xF7u);
}
__device__ __forceinline__ float group_scale(uint32_t byte) { return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7))); }
// Eight values of a group with its scale byte, in 4 bits.  A quotient, not a product with 1 / s: many values of a group lie on a
// tie between two codes.
__device__ __forceinline__ uint32_t eight_e2m1(const float (&x)[8], uint32_t byte) {
    const float scale = group_scale(byte);
    auto over = [&](float v) { return byte ? __fdiv_rn(v, scale) : copysignf(0.f, v); };
    uint32_t b = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        b |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(over(x[2 * j]), over(x[2 * j + 1])), __NV_E2M1, cudaRoundNearest)) << 8 * j;
    return b;
}
// The largest finite magnitude of eight values, and whether one is NaN.
__device__ __forceinline__ float finite_top(const float (&x)[8], bool &nan) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (fabsf(x[j]) < INFINITY) top = fmaxf(top, fabsf(x[j]));
        nan |= x[j] != x[j];
    }
    return top;
}

// One CTA per token; rows are its q heads, then k heads, then v heads.  A lane holds 8 elements of a row's lower
// half and the 8 they are rotated with, so the rotation needs no exchange: with one 16-byte piece per lane, whose
// partner is half a row of lanes away, the kernel was bound by its instructions (8 prompts of up to 4096 tokens, 64
// and 8 heads: 49 us).
template <int kDim, int kType>
__global__ void __launch_bounds__(kAppendThreads, 5) kv_append_kernel(const AppendArgs a) {
    constexpr bool kE4m3 = kType == BD_KV_E4M3;
    constexpr int kLanes = kDim / 16;  // lanes of one row
    constexpr int kRowsPerPass = kAppendThreads / kLanes;
    pdl_trigger_and_wait();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
    const int q_rows = a.q ? a.q_heads : 0;
    const int rows = q_rows + 2 * a.kv_heads;
    uint4 in[kAppendAtOnce][2];
    auto load = [&](int r0) {  // rows r0, r0 + kRowsPerPass, ..: this lane's two pieces of each
#pragma unroll
        for (int u = 0; u < kAppendAtOnce; ++u) {
            const int r = r0 + u * kRowsPerPass;
            in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
            if (r >= rows) continue;
            const bool is_v = r >= q_rows + a.kv_heads;
            if (!in_bounds(r >= 0 && r < q_rows + 2 * a.kv_heads, a.status)) continue;
            const uint8_t *src = r < q_rows ? a.q + (t * a.q_heads + r) * (kDim * 2)
                                            : (is_v ? a.v : a.k) + (t * a.kv_heads + r - q_rows - (is_v ? a.kv_heads : 0)) * (kDim * 2);
            in[u][0] = ldg_plain(src + lane * 16);
            in[u][1] = ldg_plain(src + kDim + lane * 16);
        }
    };
    load(row0);  // under way while the position and the page are looked up
    const int32_t pos = a.positions[t];
    if (pos < 0) return;  // padding
    const int64_t seq = a.seq_ids ? a.seq_ids[t] : t;
    const int64_t page_at = pos / a.page_size;
    const int slot = pos % a.page_size;
    int64_t page = -1;
    if (seq >= 0 && seq < a.n_seqs && page_at < a.max_pages && (a.rope == nullptr || pos < a.rope_len))
        page = a.page_table[seq * a.max_pages + page_at];
    if (page < 0 || page >= a.n_pages) {
        if (threadIdx.x == 0) flag_status(a.status, kDevBadIndex);
        return;
    }
    float c[8] = {}, s[8] = {};
    if (a.rope != nullptr) {
        const float *r = a.rope + pos * static_cast<int64_t>(kDim) + lane * 8;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 cv = __ldg(reinterpret_cast<const float4 *>(r + j));
            const float4 sv = __ldg(reinterpret_cast<const float4 *>(r + kDim / 2 + j));
            c[j] = cv.x, c[j + 1] = cv.y, c[j + 2] = cv.z, c[j + 3] = cv.w;
            s[j] = sv.x, s[j + 1] = sv.y, s[j + 2] = sv.z, s[j + 3] = sv.w;
        }
    }
    const int64_t slot_row = page * a.kv_heads * a.page_size + slot;
    for (int r0 = row0; r0 - row0 < rows; r0 += kAppendAtOnce * kRowsPerPass) {  // as often for every lane: maxima are shuffled
        if (r0 != row0) load(r0);
#pragma unroll
        for (int u = 0; u < kAppendAtOnce; ++u) {
            const int r = r0 + u * kRowsPerPass;
            const bool is_q = r < q_rows, is_v = r >= q_rows + a.kv_heads;
            float x[8], y[8];
            unpack8(in[u][0], x);
            unpack8(in[u][1], y);
            if (a.rope != nullptr && !is_v) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float low = __fsub_rn(__fmul_rn(x[j], c[j]), __fmul_rn(y[j], s[j]));
                    y[j] = __fadd_rn(__fmul_rn(y[j], c[j]), __fmul_rn(x[j], s[j]));
                    x[j] = low;
                }
            }
            if (is_q && in_bounds(r < a.q_heads, a.status)) {
                uint8_t *dst = a.q_out + (t * a.q_heads + r) * (kDim * 2) + lane * 16;
                *reinterpret_cast<uint4 *>(dst) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + kDim) = pack8(y);
            }
            if (__all_sync(0xFFFFFFFFu, is_q || r >= rows)) continue;
            float top = 0.f;
            if constexpr (kE4m3) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // neither infinity nor NaN
                    if (fabsf(x[j]) < INFINITY) top = fmaxf(top, fabsf(x[j]));
                    if (fabsf(y[j]) < INFINITY) top = fmaxf(top, fabsf(y[j]));
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            }
            [[maybe_unused]] float top_y = 0.f;
            [[maybe_unused]] int nan = 0;  // of the group in the lower half, and in the upper
            if constexpr (kType == BD_KV_E2M1) {  // a group is two lanes' pieces of one half
                bool n0 = false, n1 = false;
                top = finite_top(x, n0), top_y = finite_top(y, n1);
                nan = (n0 ? 1 : 0) | (n1 ? 2 : 0);
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top_y = fmaxf(top_y, __shfl_xor_sync(0xFFFFFFFFu, top_y, 1));
                nan |= __shfl_xor_sync(0xFFFFFFFFu, nan, 1);
            }
            if (is_q || r >= rows) continue;
            const int64_t at = slot_row + static_cast<int64_t>(r - q_rows - (is_v ? a.kv_heads : 0)) * a.page_size;
            if (!in_bounds(at >= 0 && at < a.n_pages * a.kv_heads * a.page_size, a.status)) continue;
            uint8_t *dst = is_v ? a.cv : a.ck;
            if constexpr (kType == BD_KV_BF16) {
                *reinterpret_cast<uint4 *>(dst + at * (kDim * 2) + lane * 16) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + at * (kDim * 2) + kDim + lane * 16) = pack8(y);
            } else if constexpr (kType == BD_KV_E2M1) {
                const uint32_t low = group_scale_byte(top), high = group_scale_byte(top_y);
                *reinterpret_cast<uint32_t *>(dst + at * (kDim / 2) + lane * 4) = eight_e2m1(x, low);
                *reinterpret_cast<uint32_t *>(dst + at * (kDim / 2) + kDim / 4 + lane * 4) = eight_e2m1(y, high);
                if (lane % 2 == 0) {
                    uint8_t *sc = (is_v ? a.cv_scale : a.ck_scale) + at * (kDim / 16) + lane / 2;
                    sc[0] = static_cast<uint8_t>(nan & 1 ? 0xFFu : low), sc[kDim / 32] = static_cast<uint8_t>(nan & 2 ? 0xFFu : high);
                }
            } else {
                const int e = scale_byte(top);
                const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e), exact
                auto eight = [&](const float (&v)[8]) {
                    uint32_t b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        b[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * j] * inv, v[2 * j + 1] * inv), __NV_SATFINITE,
                                                        __NV_E4M3);
                    return make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
                };
                *reinterpret_cast<uint2 *>(dst + at * kDim + lane * 8) = eight(x);
                *reinterpret_cast<uint2 *>(dst + at * kDim + kDim / 2 + lane * 8) = eight(y);
                if (lane == 0) (is_v ? a.cv_scale : a.ck_scale)[at] = static_cast<uint8_t>(e);
            }
        }
    }
}

// The same for a rotation of part of a head or of neighbours.  A lane holds 16 neighbouring elements, a group of the 4-bit
// cache, whatever the parts: what an element is rotated with is read a second time, from L1, where it is not among the lane's own.  Its rows are
// read before any row of the pass is written: the query may be rotated in place, and a row's lanes are one warp's.
constexpr int kGroupAtOnce = 2;

struct GroupArgs : AppendArgs {
    int32_t rope_dim, interleaved;
};

template <int kDim, int kType>
__global__ void __launch_bounds__(kAppendThreads) kv_append_group_kernel(const GroupArgs a) {
    constexpr int kLanes = kDim / 16;  // lanes of one row
    constexpr int kRowsPerPass = kAppendThreads / kLanes;
    pdl_trigger_and_wait();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
    const int q_rows = a.q ? a.q_heads : 0;
    const int rows = q_rows + 2 * a.kv_heads;
    const int half = a.rope ? a.rope_dim / 2 : 0;
    const bool turn = lane * 16 < 2 * half;  // a multiple of 16: all 16 elements or none
    const bool exchange = turn && !a.interleaved;
    uint4 in[kGroupAtOnce][2], with[kGroupAtOnce][2];
    // piece w of this lane starts at element lane * 16 + 8 w; it is rotated with the piece at partner(w)
    auto partner = [&](int w) {
        const int e = lane * 16 + 8 * w;
        return e < half ? e + half : e - half;
    };
    auto load = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kGroupAtOnce; ++u) {
            const int r = r0 + u * kRowsPerPass;
            in[u][0] = in[u][1] = with[u][0] = with[u][1] = make_uint4(0, 0, 0, 0);
            if (r >= rows) continue;
            const bool is_v = r >= q_rows + a.kv_heads;
            if (!in_bounds(r >= 0 && r < q_rows + 2 * a.kv_heads, a.status)) continue;
            const uint8_t *src = r < q_rows ? a.q + (t * a.q_heads + r) * (kDim * 2)
                                            : (is_v ? a.v : a.k) + (t * a.kv_heads + r - q_rows - (is_v ? a.kv_heads : 0)) * (kDim * 2);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                in[u][w] = ldg_plain(src + lane * 32 + w * 16);
                if (exchange && !is_v) with[u][w] = ldg_plain(src + partner(w) * 2);
            }
        }
    };
    load(row0);
    const int32_t pos = a.positions[t];
    if (pos < 0) return;  // padding
    const int64_t seq = a.seq_ids ? a.seq_ids[t] : t;
    const int64_t page_at = pos / a.page_size;
    const int slot = pos % a.page_size;
    int64_t page = -1;
    if (seq >= 0 && seq < a.n_seqs && page_at < a.max_pages && (a.rope == nullptr || pos < a.rope_len))
        page = a.page_table[seq * a.max_pages + page_at];
    if (page < 0 || page >= a.n_pages) {
        if (threadIdx.x == 0) flag_status(a.status, kDevBadIndex);
        return;
    }
    // cosines and sines: of each element where halves are exchanged, of each pair (in the first 4) where neighbours are
    float c[2][8] = {}, s[2][8] = {};
    if (turn) {
        const float *row = a.rope + pos * static_cast<int64_t>(a.rope_dim);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int e = lane * 16 + 8 * w;
            const int at = a.interleaved ? e / 2 : (e < half ? e : e - half);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                if (a.interleaved && j) continue;
                const float4 cv = __ldg(reinterpret_cast<const float4 *>(row + at + j));
                const float4 sv = __ldg(reinterpret_cast<const float4 *>(row + half + at + j));
                c[w][j] = cv.x, c[w][j + 1] = cv.y, c[w][j + 2] = cv.z, c[w][j + 3] = cv.w;
                s[w][j] = sv.x, s[w][j + 1] = sv.y, s[w][j + 2] = sv.z, s[w][j + 3] = sv.w;
            }
        }
    }
    const int64_t slot_row = page * a.kv_heads * a.page_size + slot;
    for (int r0 = row0; r0 - row0 < rows; r0 += kGroupAtOnce * kRowsPerPass) {  // as often for every lane: see the shuffles
        if (r0 != row0) load(r0);
        __syncwarp();  // what the row's other lanes read of it is read
#pragma unroll
        for (int u = 0; u < kGroupAtOnce; ++u) {
            const int r = r0 + u * kRowsPerPass;
            const bool is_q = r < q_rows, is_v = r >= q_rows + a.kv_heads;
            float x[2][8];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                unpack8(in[u][w], x[w]);
                if (!turn || is_v) continue;
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float lo = x[w][2 * j], hi = x[w][2 * j + 1];
                        x[w][2 * j] = __fsub_rn(__fmul_rn(lo, c[w][j]), __fmul_rn(hi, s[w][j]));
                        x[w][2 * j + 1] = __fadd_rn(__fmul_rn(hi, c[w][j]), __fmul_rn(lo, s[w][j]));
                    }
                } else {
                    float y[8];
                    unpack8(with[u][w], y);
                    const bool low = lane * 16 + 8 * w < half;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[w][j] = low ? __fsub_rn(__fmul_rn(x[w][j], c[w][j]), __fmul_rn(y[j], s[w][j]))
                                      : __fadd_rn(__fmul_rn(x[w][j], c[w][j]), __fmul_rn(y[j], s[w][j]));
                }
            }
            if (is_q && in_bounds(r < a.q_heads, a.status)) {
                uint4 *dst = reinterpret_cast<uint4 *>(a.q_out + (t * a.q_heads + r) * (kDim * 2) + lane * 32);
                dst[0] = pack8(x[0]), dst[1] = pack8(x[1]);
            }
            if (__all_sync(0xFFFFFFFFu, is_q || r >= rows)) continue;
            bool nan = false;
            float top = 0.f;
            if constexpr (kType != BD_KV_BF16) top = fmaxf(finite_top(x[0], nan), finite_top(x[1], nan));
            if constexpr (kType == BD_KV_E4M3) {  // a scale for the whole row
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            }
            if (is_q || r >= rows) continue;
            const int64_t at = slot_row + static_cast<int64_t>(r - q_rows - (is_v ? a.kv_heads : 0)) * a.page_size;
            if (!in_bounds(at >= 0 && at < a.n_pages * a.kv_heads * a.page_size, a.status)) continue;
            uint8_t *dst = is_v ? a.cv : a.ck, *scales = is_v ? a.cv_scale : a.ck_scale;
            if constexpr (kType == BD_KV_BF16) {
                uint4 *d = reinterpret_cast<uint4 *>(dst + at * (kDim * 2) + lane * 32);
                d[0] = pack8(x[0]), d[1] = pack8(x[1]);
            } else if constexpr (kType == BD_KV_E4M3) {
                const int e = scale_byte(top);
                const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e), exact
                uint32_t b[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    b[j] = __nv_cvt_float2_to_fp8x2(make_float2(x[j / 4][j % 4 * 2] * inv, x[j / 4][j % 4 * 2 + 1] * inv), __NV_SATFINITE,
                                                    __NV_E4M3);
                *reinterpret_cast<uint4 *>(dst + at * kDim + lane * 16) =
                    make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
                if (lane == 0) scales[at] = static_cast<uint8_t>(e);
            } else {
                const uint32_t byte = group_scale_byte(top);
                *reinterpret_cast<uint2 *>(dst + at * (kDim / 2) + lane * 8) = make_uint2(eight_e2m1(x[0], byte), eight_e2m1(x[1], byte));
                scales[at * (kDim / 16) + lane] = static_cast<uint8_t>(nan ? 0xFFu : byte);
            }
        }
    }
}

// ---- read ------------------------------------------------------------------------------

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 16;  // output rows of one CTA, at most
constexpr int kReadAtOnce = 4;   // chunks of K and of V in flight per thread

struct ReadArgs {
    const uint8_t *ck, *cv, *ck_scale, *cv_scale;
    const int32_t *page_table, *offsets;
    uint8_t *k_out, *v_out;
    unsigned *status;
    int64_t n_pages, total;
    int32_t kv_heads, page_size, n_seqs, max_pages, tokens;  // tokens: output rows of one CTA
    uint32_t per_token, magic;  // 16-byte pieces of a token's row in k_out (8 at least), and ceil(2^32 / that)
};

// Two e4m3 values times 2^(e - 127), as a bf16 pair (exact down to bf16's subnormals).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two, float scale) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return pack_bf16x2(f.x * scale, f.y * scale);
}

// Four bytes of 4-bit values times a scale, as bf16 pairs: 2 significant bits times 4 at most, exact.
__device__ __forceinline__ uint4 e2m1x8_to_bf16x8(uint32_t eight, float scale) {
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(eight >> 8 * j & 0xFFu), __NV_E2M1);
        const float2 f = __half22float2(__half2(h));
        out[j] = pack_bf16x2(f.x * scale, f.y * scale);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int kDim, int kType>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a) {
    constexpr int kChunk = kDim / 8;  // 8 elements: 16 bytes of the output
    constexpr bool kE4m3 = kType == BD_KV_E4M3;
    using Raw = typename std::conditional<kE4m3, uint2, typename std::conditional<kType == BD_KV_E2M1, uint32_t, uint4>::type>::type;
    __shared__ int64_t first[kReadTokens];                // (page * kv_heads) * page_size + slot; -1: nothing, -2: zeros
    pdl_trigger_and_wait();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
    if (static_cast<int>(threadIdx.x) < a.tokens) {
        const int64_t t = t0 + threadIdx.x;
        int64_t at = -1;
        if (t < a.total && t < a.offsets[a.n_seqs]) {
            int lo = 0, hi = a.n_seqs;  // the last sequence that starts at or before t
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (a.offsets[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int64_t pos = t - a.offsets[lo];
            const int64_t p = pos / a.page_size;
            const int64_t page = pos >= 0 && p < a.max_pages ? a.page_table[static_cast<int64_t>(lo) * a.max_pages + p] : -1;
            at = page >= 0 && page < a.n_pages ? page * a.kv_heads * a.page_size + pos % a.page_size : -2;
            if (at == -2) flag_status(a.status, kDevBadIndex);
        }
        first[threadIdx.x] = at;
    }
    __syncthreads();
    const uint32_t items = a.tokens * a.per_token;
    for (uint32_t i0 = threadIdx.x; i0 < items; i0 += kReadAtOnce * kReadThreads) {
        Raw v[kReadAtOnce][2];
        float s[kReadAtOnce][2];
        int64_t to[kReadAtOnce];
#pragma unroll
        for (int u = 0; u < kReadAtOnce; ++u) {
            const uint32_t i = i0 + u * kReadThreads;
            to[u] = -1;
            if (i >= items) continue;
            const uint32_t tok = __umulhi(i, a.magic), rest = i - tok * a.per_token;
            const int64_t f = first[tok];
            if (f == -1) continue;
            to[u] = (t0 + tok) * a.per_token + rest;
            const int64_t row = f + static_cast<int64_t>(rest / kChunk) * a.page_size;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                v[u][w] = Raw{};
                s[u][w] = 0.f;
                if (f < 0 || !in_bounds(row < a.n_pages * a.kv_heads * a.page_size, a.status)) continue;
                v[u][w] = __ldcs(reinterpret_cast<const Raw *>(w ? a.cv : a.ck) + row * kChunk + rest % kChunk);
                if constexpr (kE4m3) s[u][w] = __uint_as_float(static_cast<uint32_t>((w ? a.cv_scale : a.ck_scale)[row]) << 23);
                if constexpr (kType == BD_KV_E2M1)
                    s[u][w] = group_scale((w ? a.cv_scale : a.ck_scale)[row * (kDim / 16) + rest % kChunk / 2]);
            }
        }
#pragma unroll
        for (int u = 0; u < kReadAtOnce; ++u) {
            if (to[u] < 0 || !in_bounds(to[u] < a.total * a.per_token, a.status)) continue;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint4 *d = reinterpret_cast<uint4 *>(w ? a.v_out : a.k_out) + to[u];
                const Raw x = v[u][w];
                if constexpr (kType == BD_KV_BF16) {
                    *d = x;
                } else if constexpr (kType == BD_KV_E2M1) {
                    *d = e2m1x8_to_bf16x8(x, s[u][w]);
                } else {
                    const float f = s[u][w];
                    *d = make_uint4(e4m3x2_to_bf16x2(x.x & 0xFFFFu, f), e4m3x2_to_bf16x2(x.x >> 16, f),
                                    e4m3x2_to_bf16x2(x.y & 0xFFFFu, f), e4m3x2_to_bf16x2(x.y >> 16, f));
                }
            }
        }
    }
}

template <class Args>
cudaError_t launch_pdl(void (*kernel)(const Args), int64_t grid, int threads, const Args &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kDim>
cudaError_t launch_append(int type, int64_t n, const AppendArgs &a, cudaStream_t stream) {
    return launch_pdl(type == BD_KV_E2M1   ? kv_append_kernel<kDim, BD_KV_E2M1>
                      : type == BD_KV_E4M3 ? kv_append_kernel<kDim, BD_KV_E4M3>
                                           : kv_append_kernel<kDim, BD_KV_BF16>,
                      n, kAppendThreads, a, stream);
}
template <int kDim>
cudaError_t launch_append_group(int type, int64_t n, const GroupArgs &a, cudaStream_t stream) {
    return launch_pdl(type == BD_KV_E2M1   ? kv_append_group_kernel<kDim, BD_KV_E2M1>
                      : type == BD_KV_E4M3 ? kv_append_group_kernel<kDim, BD_KV_E4M3>
                                           : kv_append_group_kernel<kDim, BD_KV_BF16>,
                      n, kAppendThreads, a, stream);
}

}  // namespace

cudaError_t launch_kv_append(const bd_kv_cache &c, const void *q, int32_t q_heads, const void *k, const void *v,
                             int64_t n_tokens, const int32_t *seq_ids, const int32_t *positions,
                             const int32_t *page_table, int32_t n_seqs, int32_t max_pages, const float *rope,
                             int64_t rope_len, int32_t rope_dim, int32_t interleaved, void *q_out, const DevCtx &ctx,
                             cudaStream_t stream) {
    GroupArgs a;
    a.rope_dim = rope_dim;
    a.interleaved = interleaved;
    a.q = static_cast<const uint8_t *>(q);
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.q_out = static_cast<uint8_t *>(q_out);
    a.ck = static_cast<uint8_t *>(c.k);
    a.cv = static_cast<uint8_t *>(c.v);
    a.ck_scale = c.k_scale;
    a.cv_scale = c.v_scale;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.page_table = page_table;
    a.rope = rope;
    a.status = ctx.status;
    a.rope_len = rope_len;
    a.n_pages = c.n_pages;
    a.q_heads = q_heads;
    a.kv_heads = c.kv_heads;
    a.page_size = c.page_size;
    a.n_seqs = n_seqs;
    a.max_pages = max_pages;
    if (rope && (interleaved || rope_dim != c.head_dim))
        return c.head_dim == 128 ? launch_append_group<128>(c.kv_type, n_tokens, a, stream) : launch_append_group<64>(c.kv_type, n_tokens, a, stream);
    return c.head_dim == 128 ? launch_append<128>(c.kv_type, n_tokens, a, stream) : launch_append<64>(c.kv_type, n_tokens, a, stream);
}

cudaError_t launch_kv_read(const bd_kv_cache &c, const int32_t *page_table, int32_t n_seqs, int32_t max_pages,
                           const int32_t *offsets, int64_t total, void *k_out, void *v_out, const DevCtx &ctx,
                           cudaStream_t stream) {
    ReadArgs a;
    a.ck = static_cast<const uint8_t *>(c.k);
    a.cv = static_cast<const uint8_t *>(c.v);
    a.ck_scale = c.k_scale;
    a.cv_scale = c.v_scale;
    a.page_table = page_table;
    a.offsets = offsets;
    a.k_out = static_cast<uint8_t *>(k_out);
    a.v_out = static_cast<uint8_t *>(v_out);
    a.status = ctx.status;
    a.n_pages = c.n_pages;
    a.total = total;
    a.kv_heads = c.kv_heads;
    a.page_size = c.page_size;
    a.n_seqs = n_seqs;
    a.max_pages = max_pages;
    // 16 tokens a CTA, fewer where they would leave SMs without one
    a.tokens = kReadTokens;
    while (a.tokens > 1 && (total + a.tokens - 1) / a.tokens < 4 * ctx.num_sms) a.tokens /= 2;
    a.per_token = static_cast<uint32_t>(c.kv_heads * (c.head_dim / 8));
    a.magic = static_cast<uint32_t>(((uint64_t{1} << 32) + a.per_token - 1) / a.per_token);  // exact for 16 x 16384 pieces
    const int64_t grid = (total + a.tokens - 1) / a.tokens;
    const bool e = c.kv_type == BD_KV_E4M3, wide = c.head_dim == 128;
    if (c.kv_type == BD_KV_E2M1)
        return launch_pdl(wide ? kv_read_kernel<128, BD_KV_E2M1> : kv_read_kernel<64, BD_KV_E2M1>, grid, kReadThreads, a, stream);
    if (wide)
        return launch_pdl(e ? kv_read_kernel<128, BD_KV_E4M3> : kv_read_kernel<128, BD_KV_BF16>, grid, kReadThreads, a, stream);
    return launch_pdl(e ? kv_read_kernel<64, BD_KV_E4M3> : kv_read_kernel<64, BD_KV_BF16>, grid, kReadThreads, a, stream);
}

}  // namespace bd
