// sample.cu -- draw of the next token of each row: temperature, top-k, top-p,
// min-p and the Gumbel maximum over what they keep.
//
//   z_i = (x_i - M) / T,  w_i = exp(z_i),  id = argmax over kept of z_i + g_i
//
// Bound: HBM for many rows (the logits once, the noise at kept tokens), latency
// for one.  A row belongs to a cluster of CTAs with a slice of it each.  A slice is
// read again out of L2 where a filter needs that: holding it in shared memory between
// left room for two CTAs per SM only, and a row is a chain of short steps with cluster
// barriers between them that other rows' CTAs have to fill.  The passes are short
// loops: unrolled over a row in registers they were bound by fetching their code.
//
// The first pass takes the largest logit and the sum of weights relative to it, and
// draws from an unfiltered row, to within rounding (see `open`).  The filters are a
// threshold in the order (x descending, index ascending), found without sorting:
//  1. Tokens that cannot be kept are left out.  top-k: the k-th of the cluster's largest
//     thread maxima is reached by k tokens, and by few more.  top-p: tokens with t = -z above
//     ln(V / ((1 - p) sum w)) weigh less than (1 - p) sum w together, so the prefix
//     ends before them.
//  2. A histogram over t holds each bin's weight, and for top-k its count.  Every CTA adds
//     up the cluster's bins and scans them, and finds the bin that the k-th token or the
//     share p falls into.  top-k has packed its few tokens into shared memory before;
//     top-p counts what may be most of the row as it reads it, and keeps each thread's best
//     draw.  The best of these is the answer if it lies before that bin, which it does
//     with about probability p; else the threads that had a better one look again.
//  3. For top-k, and where the answer may lie in that very bin, the bin's tokens (for top-k
//     all bins up to it, if those are few; as used, all that step 1 leaves, without a
//     histogram) are sent to every CTA and ordered exactly.  A bin
//     with too many tokens is split again, by the remaining bits of t, then by the bits of
//     (x, index), which differ for any two.
// Measured, rows of 128256 fp32 logits, each call on other logits than the one before: one row with top-k and top-p
// (bf16) 12.8 us, a chain of latencies; 256 rows unfiltered 65 us (4.0 TB/s), top-k 65, top-p 140, min-p 41, greedy 37,
// of every kind 90 (77 on the same logits, of which L2 keeps a part).
//
// Sums of weights do not depend on the order of atomics: they are whole numbers.  Within a
// bin of width d, w = exp(-start) w' with w' in [1 - d, 1], and a bin sums
// round((w' - 1 + d) P / d) in 32 bits beside its count, P = 65535 or what a long slice
// leaves room for; top-p's first histogram, which needs no counts, sums parts of 2^-22 in two words (Bins::add).
// Across bins weights are fixed-point with 40 fractional bits.  The sum of all weights is
// fp32 in an order fixed by the shape.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "bd_device.cuh"
#include "bd_internal.h"

namespace bd {
namespace {

constexpr int kThreads = 512;
constexpr int kCtasPerSm = 2;     // by registers
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;   // one per thread
constexpr int kBits = 9;          // a digit: one bin
constexpr int kCap = kBins;       // tokens ordered exactly: a list is scanned as the bins are
constexpr int kIndexBits = 18;    // BD_SAMPLE_MAX_VOCAB = 2^18
constexpr int kMaxCluster = 8;
constexpr int kTops = 256;        // thread maxima from which top-k's bound is taken: two of every warp of the largest cluster
constexpr float kRange = 31.5f;   // weights below exp(-31.5) of the largest count as 0 in a prefix's sum
constexpr float kFixed = 1099511627776.f;  // 2^40
constexpr float kLog2e = 1.44269504088896f;
constexpr float kInRange = 65536.f;  // logits over T, in base 2, whose weights relative to one another are summed as they come

using u64 = unsigned long long;

struct SampleArgs {
    const uint8_t *logits;
    const float *temperature, *top_p, *min_p, *noise;
    const int32_t *top_k;
    int32_t *ids;
    float *logprob;
    unsigned *status;
    int64_t m;
    int32_t vocab, slice_units;  // 16-byte units of logits in a CTA's slice
    int32_t sorted;              // long rows are taken first
    float parts;                 // of a bin's width: what all tokens of a slice add up to still fits 32 bits
    int32_t most;                // tokens that may be kept for which there is room; with more the passes go over the slice
};

struct alignas(16) Shared {
    uint32_t count[kBins], parts[kBins];  // apart: side by side they would share half of the banks
    u64 list_order[kCap], list_mass[kCap], sorted_mass[kCap];
    uint32_t tops[kTops];
    u64 warp_mass[kWarps], warp_parts[2][kWarps];
    uint32_t warp_count[kWarps];
    float warp_value[4][kWarps];
    // written by the cluster's CTAs
    struct Rank {
        float top, sum, draw, noise;
        uint32_t n;
        u64 best, in[2], rest[2];
    } ranks[kMaxCluster];
    alignas(16) uint32_t all_tops[kTops];
    // written by one thread for its CTA
    u64 before_mass, kept_mass, threshold;
    uint32_t before_count, here, list_n, maybe_n, first, bound;
    int found;
};

// ---- cluster shared memory ----------------------------------------------------------
__device__ __forceinline__ void cluster_sync_all() {
    __syncthreads();  // the barrier's instructions want converged warps
    cluster_arrive_release();
    cluster_wait_acquire();
}
__device__ __forceinline__ uint32_t remote(const void *p, int rank) { return mapa_rank(smem_u32(p), rank); }
__device__ __forceinline__ void st_remote(uint32_t at, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t at, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t at, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_remote(uint32_t at, uint32_t v) {  // what was there before
    uint32_t before;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(before) : "r"(at), "r"(v) : "memory");
    return before;
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return static_cast<int>(r);
}

// ---- order and weight -------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Bits that ascend with the value (no NaN), and back.
__device__ __forceinline__ uint32_t ascending(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);  // -0 to +0
    return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t a) {
    return __uint_as_float(a ^ (a >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
// Smaller = earlier: larger logit first, then lower index.
__device__ __forceinline__ u64 order_of(float x, int i) {
    return static_cast<u64>(~ascending(x)) << kIndexBits | static_cast<unsigned>(i);
}
struct Row {
    float top, inv_t;
    // -z, at least 0; infinite where the weight is 0
    __device__ __forceinline__ float t_of(float x) const {
        // the largest logit gives 0 also where top or inv_t is infinite
        return x == top ? 0.f : fminf(__fmul_rn(__fsub_rn(top, x), inv_t), INFINITY);
    }
};
// Bins of equal width around multiples of it, up to t = range; the last one takes everything beyond and weighs nothing.
// Whole numbers come from adding 2^23, which leaves them in a sum's low bits: conversions have an eighth of that rate.
struct Bins {
    static constexpr float kWhole = 8388608.f;  // 2^23
    float scale, width, unit, parts_of, most;  // 1 / width, width, parts / width, its inverse, parts
    float width2;                              // of add()
    __device__ __forceinline__ Bins(float range, float parts)
        : scale((kBins - 2) / range), width(range / (kBins - 2)), unit(parts * scale), parts_of(width / parts), most(parts),
          width2(width * kLog2e) {}
    static __device__ __forceinline__ int whole(float sum) { return __float_as_int(sum) - __float_as_int(kWhole); }  // sum = 2^23 + n
    __device__ __forceinline__ int bin(float t) const { return min(whole(fmaf(t, scale, kWhole)), kBins - 1); }
    __device__ __forceinline__ float start(int b) const { return (b - 0.5f) * width; }
    __device__ __forceinline__ int sub(float t, int b) const {  // the same again within a bin
        return b == kBins - 1 ? 0 : min(max(static_cast<int>((t * scale - b + 0.5f) * kBins), 0), kBins - 1);
    }
    __device__ __forceinline__ uint32_t part(float t, int b) const {
        return b == kBins - 1 ? 0u : __float2uint_rn(fminf(fmaxf(ex2((start(b) - t) * kLog2e) - (1.f - width), 0.f) * unit, most));
    }
    // fp32 from whole numbers: the same on every CTA, 2^-22 of the weight
    __device__ __forceinline__ u64 mass(int b, uint32_t count, u64 parts) const {
        if (b == kBins - 1) return 0;
        const float w = fmaf(static_cast<float>(parts), parts_of, static_cast<float>(count) * (1.f - width));
        return __float2ull_rn(w * (ex2(start(b) * -kLog2e) * kFixed));
    }
    // Adds a token to bins that hold a weight's whole part of exp(-b width) 2^-22 in two words, its upper bits in one and
    // the lower kLow in the other, and no count: two words that 2^18 tokens do not fill.  (One word has room for 14 to 16
    // bits of a weight only: a prefix of two or three heavy tokens then ends one token too early or late.)
    static constexpr int kLow = 11;
    static constexpr float kOne = 4194304.f;  // 2^22
    __device__ __forceinline__ void add(uint32_t *high, uint32_t *low, float t) const {
        const float at = fmaf(t, scale, kWhole);
        const int b = whole(at);
        const float w = ex2(fmaf(at - kWhole, width2, t * -kLog2e));  // exp(-width / 2) .. exp(width / 2) < 1.04
        const uint32_t n = static_cast<uint32_t>(whole(fmaf(w, kOne, kWhole)));
        if (b < kBins - 1) atomicAdd(&high[b], n >> kLow), atomicAdd(&low[b], n & ((1u << kLow) - 1));
    }
    __device__ __forceinline__ u64 mass_of(int b, u64 parts) const {
        return b == kBins - 1 ? 0 : __float2ull_rn(static_cast<float>(parts) * (ex2(b * -width2) * (kFixed / kOne)));
    }
};
// floor(p * mass) for 0 < p < 1, at least 1: the first token always stays
__device__ __forceinline__ u64 share_of(float p, u64 mass) {
    return max(__umul64hi(__float2ull_rz(p * 18446744073709551616.f), mass), u64{1});
}

template <bool kF32>
struct Sampler {
    static constexpr int kPer = kF32 ? 4 : 8;    // logits of a unit
    static constexpr int kAhead = kF32 ? 4 : 3;  // units of logits in flight

    Shared &s;
    const SampleArgs &a;
    float *maybe_x;      // tokens that may be kept,
    uint32_t *maybe_at;  // and which they are
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, rank = cluster_rank(), size = cluster_size();
    int64_t e0 = 0, e1 = 0, u0 = 0;  // the row's first element and the one after its last, the slice's first unit
    int base = 0, units = 0;         // token of the slice's first element, units in the slice
    int whole_from = 0, whole_to = 0;  // units that lie wholly in the row
    int tokens = 0;                  // how many may be kept
    float reach = -INFINITY;         // they have at least this logit
    Row row;

    __device__ Sampler(Shared &shared, uint8_t *data, const SampleArgs &args)
        : s(shared), a(args), maybe_x(reinterpret_cast<float *>(data)), maybe_at(reinterpret_cast<uint32_t *>(data + args.most * 4)) {}

    // ---- the slice --------------------------------------------------------------------
    static __device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }  // NaN to -inf
    __device__ __forceinline__ bool in_array(int64_t first, int n) const {  // elements of the logits, and of the noise
        return in_bounds(first >= 0 && first + n <= a.m * a.vocab, a.status);
    }
    __device__ __forceinline__ float noise_of(int64_t e) const { return in_array(e, 1) ? a.noise[e] : 0.f; }
    __device__ __forceinline__ float logit(int64_t e) const {
        if (!in_array(e, 1)) return -INFINITY;
        if constexpr (kF32) return clean(__ldg(reinterpret_cast<const float *>(a.logits) + e));
        return clean(__uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(a.logits) + e)) << 16));
    }
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[kPer]) {
        if constexpr (kF32) {
            x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
        } else {
            x[0] = bf16lo_to_f32(u.x), x[1] = bf16hi_to_f32(u.x), x[2] = bf16lo_to_f32(u.y), x[3] = bf16hi_to_f32(u.y);
            x[4] = bf16lo_to_f32(u.z), x[5] = bf16hi_to_f32(u.z), x[6] = bf16lo_to_f32(u.w), x[7] = bf16hi_to_f32(u.w);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[j] = fmaxf(x[j], -INFINITY);  // NaN to -inf; -0 is told from +0 nowhere but in order_of
    }
    static __device__ __forceinline__ float largest(const float (&x)[kPer]) {
        float m = x[0];
#pragma unroll
        for (int j = 1; j < kPer; ++j) m = fmaxf(m, x[j]);
        return m;
    }
    __device__ __forceinline__ bool inside(int i) const { return i >= whole_from && i < whole_to; }
    __device__ __forceinline__ uint4 fetch(int i) const {
        if (!in_array((u0 + i) * kPer, kPer)) return make_uint4(0, 0, 0, 0);
        uint4 v;
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(a.logits + (u0 + i) * 16));
        return v;
    }
    // x of unit i; a unit at a ragged end of the row element by element, -inf outside the row
    __device__ __forceinline__ void read(int i, bool in, const uint4 &raw, float (&x)[kPer]) const {
        if (in) {
            unpack(raw, x);
        } else {
            for (int j = 0; j < kPer; ++j) {
                const int64_t e = (u0 + i) * kPer + j;
                const float v = e >= e0 && e < e1 ? logit(e) : -INFINITY;
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (q == j) x[q] = v;
            }
        }
    }
    // f(i, x) for this thread's units of the slice, a few loads ahead (twice as many at once, or loads of a batch
    // before its use, spill and take 3 to 10% longer)
    template <class F>
    __device__ __forceinline__ void each_unit(F f) const {
        uint4 raw[kAhead];
        auto load = [&](int q, int i) { raw[q] = inside(i) ? fetch(i) : make_uint4(0, 0, 0, 0); };
#pragma unroll
        for (int q = 0; q < kAhead; ++q) load(q, tid + q * kThreads);
        for (int i0 = tid; i0 < units; i0 += kAhead * kThreads) {
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int i = i0 + q * kThreads;
                if (i >= units) break;
                float x[kPer];
                read(i, inside(i), raw[q], x);
                load(q, i + kAhead * kThreads);
                f(i, x);
            }
        }
    }
    // f(i, x, noise) for this thread's units, one ahead (two: 256 unfiltered bf16 rows 69 us, one 54)
    template <class F>
    __device__ __forceinline__ void each_scored(F f) const {
        uint4 raw;
        float next[kPer];
        auto load = [&](int i) {
            if (inside(i)) raw = fetch(i), fetch_noise(i, next);
        };
        load(tid);
        for (int i = tid; i < units; i += kThreads) {
            float x[kPer], noise[kPer];
            read(i, inside(i), raw, x);
            finish_noise(i, x, next, noise);
            load(i + kThreads);
            f(i, x, noise);
        }
    }
    __device__ __forceinline__ void fetch_noise(int i, float (&noise)[kPer]) const {
        const float *g = a.noise + (e0 + base) + static_cast<int64_t>(i) * kPer;
        if (!in_array(g - a.noise, kPer)) return;
#pragma unroll
        for (int j = 0; j < kPer; j += 4)
            asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(noise[j]), "=f"(noise[j + 1]), "=f"(noise[j + 2]), "=f"(noise[j + 3])
                         : "l"(g + j));
    }
    // the same of a unit at a ragged end, for its tokens in the row
    __device__ __forceinline__ void finish_noise(int i, const float (&x)[kPer], const float (&fetched)[kPer], float (&noise)[kPer]) const {
        if (inside(i)) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) noise[j] = fetched[j];
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                noise[j] = x[j] > -INFINITY ? noise_of(e0 + base + static_cast<int64_t>(i) * kPer + j) : 0.f;
        }
    }
    // x and noise of one unit
    __device__ __forceinline__ void read_scored(int i, float (&x)[kPer], float (&noise)[kPer]) const {
        const bool in = inside(i);
        uint4 raw = make_uint4(0, 0, 0, 0);
        float fetched[kPer];
        if (in) raw = fetch(i), fetch_noise(i, fetched);
        read(i, in, raw, x);
        finish_noise(i, x, fetched, noise);
    }
    // f(x, token) for this thread's share of the tokens that may be kept
    template <class F>
    __device__ __forceinline__ void each_token(F f) const {
        if (tokens <= a.most) {
            for (int i = tid; i < tokens; i += kThreads) f(maybe_x[i], static_cast<int>(maybe_at[i]));
        } else {
            each_unit([&](int i, const float (&x)[kPer]) {
                if (!(largest(x) >= reach)) return;
#pragma unroll 1
                for (int j = 0; j < kPer; ++j) {
                    float v = x[0];
#pragma unroll
                    for (int q = 1; q < kPer; ++q) v = q == j ? x[q] : v;
                    if (v >= reach && v > -INFINITY) f(v, base + i * kPer + j);
                }
            });
        }
    }

    template <bool kMax>
    __device__ __forceinline__ float block_fold(float v, float *smem) {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) {
            const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
            v = kMax ? fmaxf(v, u) : v + u;
        }
        if (lane == 0) smem[warp] = v;
        __syncthreads();
        float r = smem[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) r = kMax ? fmaxf(r, smem[w]) : r + smem[w];
        return r;
    }

    // ---- bins -------------------------------------------------------------------------
    // Count and weight of a thread's place (a bin, or a token of a list), and of all places up to it.
    struct Scan {
        uint32_t count, count_upto, count_all;
        u64 mass, mass_upto, mass_all;
    };
    __device__ __forceinline__ Scan scan(uint32_t count, u64 mass) {
        Scan r = {count, count, 0, mass, mass, 0};
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, r.count_upto, o);
            const u64 v = __shfl_up_sync(0xFFFFFFFFu, r.mass_upto, o);
            if (lane >= o) r.count_upto += u, r.mass_upto += v;
        }
        __syncthreads();
        if (lane == 31) s.warp_count[warp] = r.count_upto, s.warp_mass[warp] = r.mass_upto;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
            const uint32_t u = s.warp_count[q];
            const u64 v = s.warp_mass[q];
            if (q < warp) r.count_upto += u, r.mass_upto += v;
            r.count_all += u, r.mass_all += v;
        }
        return r;
    }
    // The first bin at which the count or the weight reaches `need`, what precedes it in s.before_*, its own
    // count in s.here.  Where rounding leaves the sum of all bins short, the last bin that holds a token.
    __device__ __forceinline__ int find(const Scan &c, bool by_mass, u64 need) {
        const uint32_t n = c.count_upto - c.count;
        const u64 w = c.mass_upto - c.mass;
        bool here;
        if ((by_mass ? c.mass_all : c.count_all) < need) here = c.count > 0 && c.count_upto == c.count_all;
        else here = by_mass ? c.mass_upto >= need && w < need : c.count_upto >= need && n < need;
        __syncthreads();
        if (here) s.found = tid, s.before_count = n, s.before_mass = w, s.here = c.count;
        __syncthreads();
        return s.found;
    }

    // The set of tokens chosen so far, of which a histogram tells one digit.
    struct Level {
        int depth, bin, sub, shift;
        u64 prefix;
    };
    __device__ __forceinline__ int digit_of(const Bins &bins, const Level &at, float t, u64 o) const {
        const int b = bins.bin(t);
        if (at.depth == 0) return b;
        if (b != at.bin) return -1;
        const int c = bins.sub(t, b);
        if (at.depth == 1) return c;
        if (c != at.sub || (at.depth > 2 && o >> (at.shift + kBits) != at.prefix)) return -1;
        return static_cast<int>(o >> at.shift) & (kBins - 1);
    }
    __device__ __forceinline__ void clear_bins() {
        s.count[tid] = s.parts[tid] = 0;
        __syncthreads();
    }
    __device__ void histogram(const Bins &bins, const Level &at, u64 limit) {
        clear_bins();
        each_token([&](float x, int i) {
            const float t = row.t_of(x);
            const u64 o = order_of(x, i);
            if (o > limit) return;
            const int d = digit_of(bins, at, t, o);
            if (d < 0) return;
            atomicAdd(&s.count[d], 1u);
            atomicAdd(&s.parts[d], bins.part(t, at.depth == 0 ? d : at.bin));
        });
    }
    // The cluster's totals of this thread's bin, and each CTA's count in it (four 16-bit fields a word; what is
    // gathered by them is at most kCap tokens).
    struct Each {
        u64 lo, hi;
    };
    __device__ __forceinline__ Scan totals(const Bins &bins, const Level &at, Each &each) {
        uint32_t v[kMaxCluster], w[kMaxCluster];
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            v[q] = q < size ? ld_remote(remote(&s.count[tid], q)) : 0;
            w[q] = q < size ? ld_remote(remote(&s.parts[tid], q)) : 0;
        }
        uint32_t n = 0;
        u64 parts = 0;
        each.lo = each.hi = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            n += v[q], parts += w[q];
            (q < 4 ? each.lo : each.hi) |= static_cast<u64>(min(v[q], 0xFFFFu)) << 16 * (q % 4);
        }
        return scan(n, bins.mass(at.depth == 0 ? tid : at.bin, n, parts));
    }
    __device__ __forceinline__ Scan totals_of_whole(const Bins &bins) {
        u64 parts = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q)
            if (q < size) parts += (static_cast<u64>(ld_remote(remote(&s.count[tid], q))) << Bins::kLow) + ld_remote(remote(&s.parts[tid], q));
        return scan(parts > 0, bins.mass_of(tid, parts));
    }
    // Sends this CTA's tokens of one set to every CTA's list: digit d at level `at`, or with `upto` all bins up to d.
    // The places follow from the counts that every CTA has of every other.
    __device__ void gather(const Bins &bins, const Level &at, int d, bool upto, u64 limit, const Each &each) {
        const bool mine = upto ? tid <= d : tid == d;
        u64 lo = mine ? each.lo : 0, hi = mine ? each.hi : 0;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) lo += __shfl_xor_sync(0xFFFFFFFFu, lo, o), hi += __shfl_xor_sync(0xFFFFFFFFu, hi, o);
        if (lane == 0) s.warp_parts[0][warp] = lo, s.warp_parts[1][warp] = hi;
        if (tid == 0) s.list_n = 0;
        __syncthreads();
        lo = hi = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) lo += s.warp_parts[0][w], hi += s.warp_parts[1][w];
        uint32_t first = 0;
        for (int c = 0; c < rank; ++c) first += static_cast<uint32_t>((c < 4 ? lo : hi) >> 16 * (c % 4)) & 0xFFFFu;
        each_token([&](float x, int i) {
            const float t = row.t_of(x);
            const u64 o = order_of(x, i);
            if (o > limit) return;
            const int g = digit_of(bins, at, t, o);
            if (upto ? g > d : g != d) return;
            const uint32_t slot = first + atomicAdd(&s.list_n, 1u);
            if (slot >= kCap) return;  // never: the counts say so
            const int b = bins.bin(t);
            const u64 w = bins.mass(b, 1, bins.part(t, b));
            for (int c = 0; c < size; ++c) st_remote(remote(&s.list_order[slot], c), o), st_remote(remote(&s.list_mass[slot], c), w);
        });
    }
    // Orders the n gathered tokens.  Kept are the first `need`, or by_mass those before which the weight stays below
    // `need`; with share < 1, of the first `need` those before which less than that share of their weight lies.  The
    // last kept token's order and the kept weight go to s.threshold and s.kept_mass.
    __device__ void cut(uint32_t n, bool by_mass, u64 need, float share) {
        for (int i = n + tid; i < kCap; i += kThreads) s.list_order[i] = ~0ull, s.list_mass[i] = 0, s.sorted_mass[i] = 0;
        __syncthreads();
        // ranks by counting, as many threads to a token as the list leaves
        const int lanes = n * 8 <= kThreads ? 8 : n * 4 <= kThreads ? 4 : n * 2 <= kThreads ? 2 : 1;
        const uint32_t pairs = (n + 1) / 2;
        const int i = tid / lanes, part = tid % lanes;
        const u64 mine = s.list_order[i];
        uint32_t rank_of = 0;
#pragma unroll 1
        for (uint32_t j = part; j < pairs; j += lanes) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&s.list_order[2 * j]);
            rank_of += (two.x < mine) + (two.y < mine);
        }
        if (lanes > 1) rank_of += __shfl_xor_sync(0xFFFFFFFFu, rank_of, 1);
        if (lanes > 2) rank_of += __shfl_xor_sync(0xFFFFFFFFu, rank_of, 2);
        if (lanes > 4) rank_of += __shfl_xor_sync(0xFFFFFFFFu, rank_of, 4);
        const bool on = i < n && part == 0;
        if (on) s.sorted_mass[rank_of] = s.list_mass[i];
        __syncthreads();
        // weights in that order, a place to a thread
        const u64 w = s.sorted_mass[tid];
        const Scan c = scan(tid < n, w);
        u64 end = need;
        if (share < 1.f) {
            if (tid == static_cast<uint32_t>(min(need, static_cast<u64>(n))) - 1) s.kept_mass = c.mass_upto;
            __syncthreads();
            end = share_of(share, s.kept_mass);
        }
        const bool keep = tid < n && (by_mass || static_cast<u64>(tid) < need) &&
                          (!(by_mass || share < 1.f) || c.mass_upto - w < end);
        const int kept = __syncthreads_count(keep);  // they are the first ones
        if (tid == kept - 1) s.kept_mass = c.mass_upto;
        if (on && rank_of == kept - 1) s.threshold = mine;
        __syncthreads();
    }

    // The order of the last token to keep of level-0 bin d (`here` tokens, counts by CTA in `each`): its first `need`
    // tokens, or those before which its weight stays below `need`.  `limited`: the bin's counts include tokens
    // beyond `limit`.  *kept receives the weight of the bin's kept tokens.
    __device__ u64 refine(const Bins &bins, int d, bool by_mass, u64 need, uint32_t here, Each each, u64 limit, bool limited,
                          u64 *kept) {
        Level at = {0, d, 0, 0, 0};
        int digit = d;
        *kept = 0;
        while ((here > kCap || limited) && at.depth < 7) {  // (7 digits tell any two tokens apart)
            limited = false;
            if (at.depth == 1) at.sub = digit;
            if (at.depth > 1) at.prefix = at.prefix << kBits | static_cast<unsigned>(digit);
            ++at.depth;
            at.shift = at.depth == 2 ? 32 + kIndexBits - kBits : at.shift - kBits;
            cluster_sync_all();  // nobody reads the bins any more
            histogram(bins, at, limit);
            cluster_sync_all();
            const Scan c = totals(bins, at, each);
            digit = find(c, by_mass, need);
            need -= by_mass ? s.before_mass : s.before_count;
            *kept += s.before_mass;
            here = s.here;
        }
        gather(bins, at, digit, false, limit, each);
        cluster_sync_all();
        cut(here, by_mass, need, 1.f);
        *kept += s.kept_mass;
        return s.threshold;
    }

    __device__ int64_t row_of(int64_t turn);
    __device__ void run(int64_t r);
};

// The row that the cluster of this number takes: rows with a share p alone first, as they take two to three times as
// long as others and would otherwise end last (256 rows of every kind, the same logits: 87 us in their own order, 77 so).
template <bool kF32>
__device__ int64_t Sampler<kF32>::row_of(int64_t turn) {
    if (!a.sorted) return turn;
    auto is_long = [&](int64_t r) {
        const float p = a.top_p[r];
        const int k = a.top_k ? a.top_k[r] : 0;
        return p > 0.f && p < 1.f && (k <= 0 || k >= a.vocab) && (!a.temperature || a.temperature[r] > 0.f);
    };
    int mine = 0;
    for (int64_t r = tid; r < a.m; r += kThreads) mine += is_long(r);
    const int all = __syncthreads_or(mine) ? static_cast<int>(scan(mine, 0).count_all) : 0;
    if (all == 0) return turn;
    const bool want = turn < all;
    int64_t left = want ? turn : turn - all;  // rows of this sort before the one that is wanted
    for (int64_t r0 = 0; r0 < a.m; r0 += kThreads) {
        const bool on = r0 + tid < a.m && is_long(r0 + tid) == want;
        const Scan c = scan(on, 0);
        if (left >= c.count_all) {
            left -= c.count_all;
            continue;
        }
        if (on && c.count_upto == left + 1) s.found = static_cast<int>(r0 + tid);
        __syncthreads();
        const int64_t r = s.found;
        __syncthreads();
        return r;
    }
    return turn;  // never
}

template <bool kF32>
__device__ void Sampler<kF32>::run(int64_t r) {
    // units at multiples of kPer of the whole array: 16-byte aligned logits, and 16-byte aligned noise
    e0 = r * a.vocab, e1 = e0 + a.vocab;
    u0 = e0 / kPer + static_cast<int64_t>(rank) * a.slice_units;
    units = static_cast<int>(max(min(u0 + a.slice_units, (e1 + kPer - 1) / kPer) - u0, int64_t{0}));
    base = static_cast<int>(u0 * kPer - e0);
    whole_from = base < 0 ? 1 : 0;
    whole_to = static_cast<int>(min(e1 / kPer - u0, static_cast<int64_t>(units)));
    // settings
    const float temp = a.temperature ? a.temperature[r] : 1.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    float p = a.top_p ? a.top_p[r] : 1.f;
    float low = a.min_p ? a.min_p[r] : 0.f;
    const bool greedy = !(temp > 0.f);
    row.inv_t = greedy ? 1.f : __fdiv_rn(1.f, temp);
    uint32_t k = top_k > 0 && top_k < a.vocab ? static_cast<uint32_t>(top_k) : 0;
    if (p <= 0.f) k = 1;
    if (!(p > 0.f && p < 1.f) || k == 1) p = 1.f;
    low = low > 0.f ? fminf(low, 1.f) : 0.f;
    const bool filtered = !greedy && (k > 0 || p < 1.f);
    const bool open = !greedy && !filtered && low == 0.f;
    // the noise, which top-p's second pass reads beside the logits whether or not a token is kept, is on its way into L2
    // meanwhile
    if (tid == 0 && !greedy && k == 0 && p < 1.f) {
        const int64_t n = min(static_cast<int64_t>(units), a.m * a.vocab / kPer - u0);
        if (n > 0 && in_bounds(u0 >= 0 && (u0 + n) * kPer <= a.m * a.vocab, a.status))
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.noise + u0 * kPer), "r"(static_cast<uint32_t>(n * kPer * 4))
                         : "memory");
    }

    // First pass: each thread's largest logit and the unit it is first met in, and the sum of its weights relative to
    // the largest so far, or rather to `shift`, which is that times per rounded: x per - shift is one operation.
    const float per = row.inv_t * kLog2e;
    const bool plain = per > 0.f && per < INFINITY;
    float top = -INFINITY, next_top = -INFINITY, shift = 0.f, sum = 0.f;  // next_top: the largest logit of other units
    int top_unit = 0;
    auto weigh = [&](int i, const float (&x)[kPer], auto next) {
        const float here = largest(x);
        if (here > top) {
            const float to = here * per;
            // beyond this range a sum means nothing (`shift` may be infinite, so may the sum), and any larger logit that
            // is in range outweighs it wholly
            sum = top > -INFINITY && fabsf(shift) < kInRange ? sum * ex2(shift - to) : 0.f;
            if constexpr (next) next_top = top;
            top = here, shift = to, top_unit = i;
        } else if constexpr (next) {
            next_top = fmaxf(next_top, here);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += ex2(fmaf(x[j], per, -shift));
    };
    // An unfiltered row is drawn from in the same pass: scores without M, x / T + g, are off by little, so the threads
    // that may have met the best one are known once all have, and look at it again.
    float most = -INFINITY, second = -INFINITY, loudest = -INFINITY;
    int draw_unit = -1;
    if (open)
        each_scored([&](int i, const float (&x)[kPer], const float (&noise)[kPer]) {
            weigh(i, x, std::false_type{});
            float score[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) score[j] = fmaf(x[j], row.inv_t, noise[j]);
            const float here = largest(score);
            loudest = fmaxf(loudest, largest(noise));
            if (here > most) second = most, most = here, draw_unit = i;
            else second = fmaxf(second, here);
        });
    else
        each_unit([&](int i, const float (&x)[kPer]) { weigh(i, x, std::true_type{}); });

    // This CTA's largest logit and the sum of its weights relative to it.  For top-k the largest of each warp's thread
    // maxima, kTops in the cluster, of which the k-th is a bound that k tokens reach; for a larger k each warp's j-th
    // largest, of which the smallest is one.
    const int per_warp = kTops / (size * kWarps);
    const bool by_rank = k <= kTops;
    const int sent = by_rank ? kWarps * per_warp : kWarps;  // by this CTA
    if (filtered && k > 0) {
        const uint32_t j = by_rank ? per_warp : (k + size * kWarps - 1) / (size * kWarps);
        uint32_t left = ascending(top), jth = 0;  // 0: below every logit
        if (j <= 32)
            for (uint32_t i = 0; i < j; ++i) {
                jth = __reduce_max_sync(0xFFFFFFFFu, left);
                const unsigned who = __ballot_sync(0xFFFFFFFFu, left == jth);
                if (lane == __ffs(who) - 1) left = 0;
                if (by_rank && lane == 0) s.tops[warp * per_warp + i] = jth;
            }
        if (!by_rank && lane == 0) s.tops[warp] = jth;
    }
    const float cta_top = block_fold<true>(top, s.warp_value[0]);
    if (plain && fabsf(cta_top * per) < kInRange / 2) {
        // a thread whose largest logit lies beyond the range of its own sum weighs nothing beside that
        sum = top > -INFINITY && fabsf(shift) < kInRange ? sum * ex2(fmaf(-cta_top, per, shift)) : 0.f;
    } else {  // a logit or a setting at the end of its range
        sum = 0.f;
        const Row own = {cta_top, row.inv_t};
        for (int i = tid; i < units * kPer && cta_top > -INFINITY; i += kThreads) {
            const int64_t e = u0 * kPer + i;
            const float x = e >= e0 && e < e1 ? logit(e) : -INFINITY;
            if (x > -INFINITY) sum += ex2(own.t_of(x) * -kLog2e);
        }
    }
    sum = block_fold<false>(sum, s.warp_value[1]);
    float cta_most = -INFINITY;
    if (open) cta_most = block_fold<true>(most, s.warp_value[2]), loudest = block_fold<true>(loudest, s.warp_value[3]);
    __syncwarp();
    cluster_wait_acquire();  // every CTA of the cluster runs: its shared memory may be written
    if (tid < size) {
        const uint32_t to = remote(&s.ranks[rank], tid);
        st_remote(to, cta_top), st_remote(to + 4, sum), st_remote(to + 8, cta_most), st_remote(to + 12, loudest);
    }
    if (filtered && k > 0 && tid < sent * size) {  // sent: a power of two
        const int i = tid & (sent - 1);
        st_remote(remote(&s.all_tops[rank * sent + i], tid >> (__ffs(sent) - 1)), s.tops[i]);
    }
    if (tid == 0) s.list_n = s.maybe_n = 0;
    cluster_sync_all();
    row.top = s.ranks[0].top;
    for (int c = 1; c < size; ++c) row.top = fmaxf(row.top, s.ranks[c].top);
    if (row.top == -INFINITY) {  // nothing may be drawn; the whole cluster leaves
        if (rank == 0 && tid == 0 && in_bounds(r >= 0 && r < a.m, a.status)) {
            a.ids[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        return;
    }
    float weight = 0.f;
    for (int c = 0; c < size; ++c) {
        const float v = s.ranks[c].top;
        if (v > -INFINITY) weight = fmaf(s.ranks[c].sum, ex2(row.t_of(v) * -kLog2e), weight);
    }

    // f(i, x) for the units that hold a logit of at least `bound`, and some others.  Most threads have none or one, which
    // the first pass has left; through all units of a thread with more the warp looks together, or each such thread by
    // itself where that takes no more rounds of loads.
    auto candidates = [&](float bound, auto f) {
        const bool more = next_top >= bound;
        float x[kPer];
        if (!more && top >= bound) {
            read(top_unit, inside(top_unit), inside(top_unit) ? fetch(top_unit) : make_uint4(0, 0, 0, 0), x);
            f(top_unit, x);
        }
        unsigned who = __ballot_sync(0xFFFFFFFFu, more);
        if (__popc(who) * (kAhead * kThreads) > units) {
            if (more) each_unit(f);
        } else {
            for (; who; who &= who - 1)
                for (int i = tid - lane + __ffs(who) - 1 + lane * kThreads; i < units; i += 32 * kThreads) {
                    read(i, inside(i), inside(i) ? fetch(i) : make_uint4(0, 0, 0, 0), x);
                    f(i, x);
                }
        }
    };

    u64 best = 0;
    auto offer = [&](float t, float noise, int i) {
        const float score = fmaxf(__fadd_rn(-t, fmaxf(noise, -INFINITY)), -INFINITY);
        const u64 c = static_cast<u64>(ascending(score)) << 32 | (0xFFFFFFFFu - static_cast<unsigned>(i));
        best = c > best ? c : best;
    };
    auto fold_max = [&](u64 v) {  // over the CTA
#pragma unroll
        for (int o = 16; o > 0; o /= 2) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        __syncthreads();
        if (lane == 0) s.warp_mass[warp] = v;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) v = max(v, s.warp_mass[w]);
        return v;
    };
    auto answer = [&] {  // by one thread of the cluster
        const int id = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
        if (!in_bounds(r >= 0 && r < a.m && id >= 0 && id < a.vocab, a.status)) return;
        a.ids[r] = id;
        if (a.logprob) a.logprob[r] = -row.t_of(logit(e0 + id)) - logf(weight);
    };
    auto answer_of_all = [&] {
        best = fold_max(best);
        if (tid == 0) st_remote(remote(&s.ranks[rank].best, 0), best);
        cluster_sync_all();
        if (rank == 0 && tid == 0) {
            for (int c = 0; c < size; ++c) best = s.ranks[c].best > best ? s.ranks[c].best : best;
            answer();
        }
    };
    if (greedy) {  // the first pass has met it
        if (top == row.top) {
            float x[kPer];
            read(top_unit, inside(top_unit), inside(top_unit) ? fetch(top_unit) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
            for (int j = kPer - 1; j >= 0; --j)
                if (x[j] == top) best = 1ull << 32 | (0xFFFFFFFFu - static_cast<unsigned>(base + top_unit * kPer + j));
        }
        answer_of_all();
        return;
    }
    if (open && plain && row.top < INFINITY) {
        for (int c = 0; c < size; ++c) cta_most = fmaxf(cta_most, s.ranks[c].draw), loudest = fmaxf(loudest, s.ranks[c].noise);
        // A first look is off by 2^-24 of itself, the score by that of itself and twice that of z, all of which
        // this bounds for the best of either; `least` is below the first look of the best score.
        const float size_of = fabsf(row.top * row.inv_t) + fabsf(cta_most) + fabsf(loudest);
        const bool sharp = size_of < 1e30f;  // (not with NaN)
        const float least = sharp ? cta_most - size_of * 9.5367431640625e-7f : -INFINITY;  // 2^-20
        float score = -INFINITY;
        int first = -1;  // of equal scores the one met first has the lowest index
        auto look = [&](int i, const float (&x)[kPer], const float (&noise)[kPer]) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const float v = __fadd_rn(__fmul_rn(__fsub_rn(x[j], row.top), row.inv_t), noise[j]);
                if (v > score) score = v, first = i * kPer + j;
            }
        };
        if (second >= least) {
            each_scored(look);
        } else if (most >= least && draw_unit >= 0) {
            float x[kPer], noise[kPer];
            read_scored(draw_unit, x, noise);
            look(draw_unit, x, noise);
        }
        if (first >= 0) best = static_cast<u64>(ascending(score)) << 32 | (0xFFFFFFFFu - static_cast<unsigned>(base + first));
        if (!sharp && !__syncthreads_or(first >= 0)) {  // a slice whose scores are all -inf (or NaN, which counts as -inf): its first token
            each_unit([&](int i, const float (&x)[kPer]) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (x[j] > -INFINITY) offer(INFINITY, -INFINITY, base + i * kPer + j);
            });
        }
        answer_of_all();
        return;
    }
    if (!filtered) {  // the tokens of min-p, or settings and logits at the end of their range
        // Below any token that the exact test keeps: t, logf(low) * temp and their sum with the largest logit are off
        // by less than 2^-21 of themselves, and expf(-t) by less than 2^-21.
        const float down = low > 0.f ? logf(low) * temp : -INFINITY;
        float least = plain && row.top < INFINITY ? row.top + down : -INFINITY;
        least -= (fabsf(least) + fabsf(down) + temp) * 1e-6f;
        if (!(least > -INFINITY)) least = -INFINITY;
        candidates(least, [&](int i, const float (&x)[kPer]) {
            if (largest(x) < least) return;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (x[j] == -INFINITY) continue;
                const float t = row.t_of(x[j]);
                if (low == 0.f || expf(-t) >= low) offer(t, noise_of(e0 + base + i * kPer + j), base + i * kPer + j);
            }
        });
        answer_of_all();
        return;
    }

    // tokens that may be kept: x >= reach
    float range = kRange;
    bool pruned = false;  // by weight
    if (k > 0) {
        if (warp == 0) {  // bit by bit, of the bits in which they differ
            uint32_t v[kTops / 32], bound = 0xFFFFFFFFu;
            if (by_rank) {
                uint32_t some = 0, every = 0xFFFFFFFFu;
#pragma unroll
                for (int i = 0; i < kTops / 32; ++i) v[i] = s.all_tops[lane + 32 * i], some |= v[i], every &= v[i];
                some = __reduce_or_sync(0xFFFFFFFFu, some), every = __reduce_and_sync(0xFFFFFFFFu, every);
                bound = every;
#pragma unroll 1
                for (uint32_t bits = some & ~every; bits;) {
                    const uint32_t bit = 1u << (31 - __clz(bits)), least = bound | bit;
                    bits ^= bit;
                    uint32_t reached = 0;
#pragma unroll
                    for (int i = 0; i < kTops / 32; ++i) reached += v[i] >= least;
                    if (__reduce_add_sync(0xFFFFFFFFu, reached) >= k) bound = least;
                }
            } else {
                for (int i = lane; i < sent * size; i += 32) bound = min(bound, s.all_tops[i]);
                bound = __reduce_min_sync(0xFFFFFFFFu, bound);
            }
            if (lane == 0) s.bound = bound;
        }
        __syncthreads();
        reach = s.bound > ascending(-INFINITY) ? value_of(s.bound) : -INFINITY;
        if (reach > -INFINITY) range = fminf(range, row.t_of(reach) * 1.0001f + 1e-6f);
    } else if (p < 1.f - 1e-5f) {  // a longer prefix is summed over everything, so that it ends by the sum of its own bins
        const float bound = logf(static_cast<float>(a.vocab) / ((1.f - p) * 0.99f * weight));
        if (bound < kRange && row.top < INFINITY && plain) {
            pruned = true;
            range = fmaxf(bound, 1e-3f);
            reach = row.top - range * temp;
            reach -= fabsf(reach) * 1e-6f;
            if (!(reach > -INFINITY)) reach = -INFINITY;
        }
    }
    const Bins bins(range, a.parts);
    const Level level0 = {0, 0, 0, 0, 0};
    auto keep = [&](float x, int token) {  // one more token of which the bins are told, or that is ordered
        const uint32_t place = atomicAdd(&s.maybe_n, 1u);
        if (place < a.most) maybe_x[place] = x, maybe_at[place] = static_cast<uint32_t>(token);
    };
    u64 threshold = ~0ull;
    Each each;
    if (k > 0) {  // few tokens: packed, then counted
        each_unit([&](int i, const float (&x)[kPer]) {
            if (!(largest(x) >= reach)) return;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (x[j] >= reach && x[j] > -INFINITY) keep(x[j], base + i * kPer + j);
        });
        __syncthreads();
        tokens = static_cast<int>(s.maybe_n);
        // orders a list, takes the share p, draws
        auto draw_of_list = [&](uint32_t n) {
            cut(n, false, k, p);
            for (int i = tid; i < n; i += kThreads) {
                const u64 o = s.list_order[i];
                if (o > s.threshold) continue;
                const int token = static_cast<int>(o & ((1u << kIndexBits) - 1));
                const float t = row.t_of(value_of(~static_cast<uint32_t>(o >> kIndexBits)));
                if (low == 0.f || expf(-t) >= low) offer(t, noise_of(e0 + token), token);
            }
            best = fold_max(best);
            if (tid == 0) answer();
        };
        // As used they are few: straight to the first CTA's list.
        if (tid < size) st_remote(remote(&s.ranks[rank].n, tid), static_cast<uint32_t>(tokens));
        if (tid == 0) s.first = add_remote(remote(&s.list_n, 0), static_cast<uint32_t>(min(tokens, kCap + 1)));
        __syncthreads();
        if (s.first + tokens <= kCap && tokens <= a.most)
            for (int i = tid; i < tokens; i += kThreads) {
                const float x = maybe_x[i], t = row.t_of(x);
                const int b = bins.bin(t);
                st_remote(remote(&s.list_order[s.first + i], 0), order_of(x, static_cast<int>(maybe_at[i])));
                st_remote(remote(&s.list_mass[s.first + i], 0), bins.mass(b, 1, bins.part(t, b)));
            }
        cluster_sync_all();
        uint64_t in_all = 0;
        for (int c = 0; c < size; ++c) in_all += s.ranks[c].n;
        if (in_all <= min(kCap, a.most)) {
            if (rank == 0) draw_of_list(static_cast<uint32_t>(in_all));
            return;
        }
        histogram(bins, level0, ~0ull);
        cluster_sync_all();
        const Scan c = totals(bins, level0, each);
        const int d = find(c, false, k);
        const uint32_t upto = s.before_count + s.here, need = k - min(s.before_count, k), here = s.here;
        const u64 before_mass = s.before_mass;
        if (upto <= kCap) {
            gather(bins, level0, d, true, ~0ull, each);
            cluster_sync_all();
            if (rank == 0) draw_of_list(upto);
            return;
        }
        u64 kept;
        threshold = refine(bins, d, false, need, here, each, ~0ull, false, &kept);
        if (p < 1.f) {  // the share p of what is kept: it ends in a bin before d, or in what is kept of d
            const u64 target = share_of(p, before_mass + kept);
            cluster_sync_all();  // nobody reads the list any more
            if (target <= before_mass) {
                const int d2 = find(c, true, target);
                threshold = refine(bins, d2, true, target - s.before_mass, s.here, each, ~0ull, false, &kept);
            } else {
                threshold = refine(bins, d, true, target - before_mass, here, each, threshold, true, &kept);
            }
        }
    } else {
        // The weights of bins, and each thread's best draw among tokens that may be kept.
        auto key_of = [&](float score, int i) { return static_cast<u64>(ascending(score)) << 32 | (0xFFFFFFFFu - static_cast<unsigned>(i)); };
        int unit = -1;
        clear_bins();
        auto weigh_bins = [&](auto exact) {
            each_scored([&](int i, const float (&x)[kPer], const float (&noise)[kPer]) {
                if (!(largest(x) >= reach)) return;
                float score[kPer];
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const float t = exact ? row.t_of(x[j]) : __fmul_rn(__fsub_rn(row.top, x[j]), row.inv_t);
                    score[j] = __fadd_rn(-t, noise[j]);
                    bins.add(s.count, s.parts, t);
                }
                const float here = largest(score);
                if (here > most) most = here, unit = i;
            });
        };
        if (plain && row.top < INFINITY) weigh_bins(std::false_type{});
        else weigh_bins(std::true_type{});
        cluster_sync_all();
        const Scan c = totals_of_whole(bins);
        const u64 need = share_of(p, pruned ? __float2ull_rn(weight * kFixed) : c.mass_all);
        const int d = find(c, true, need);
        const u64 need_here = need - min(s.before_mass, need - 1);
        // Of the threads' best draws those before bin d are kept.  Where one that is not (or is of bin d) would beat
        // them all, its thread looks through its tokens again; mostly none does.
        auto place = [&](float x, float &t) {  // 0: kept, 1: of bin d, 2: not kept
            t = row.t_of(x);
            const int b = bins.bin(t);
            return low > 0.f && !(expf(-t) >= low) ? 2 : b < d ? 0 : b == d ? 1 : 2;
        };
        auto exchange = [&](int round, u64 &in, u64 &rest) {
#pragma unroll
            for (int o = 16; o > 0; o /= 2) {
                in = max(in, __shfl_xor_sync(0xFFFFFFFFu, in, o));
                rest = max(rest, __shfl_xor_sync(0xFFFFFFFFu, rest, o));
            }
            __syncthreads();
            if (lane == 0) s.warp_parts[0][warp] = in, s.warp_parts[1][warp] = rest;
            __syncthreads();
            if (warp == 0 && lane < size) {
                for (int w = 0; w < kWarps; ++w) in = max(in, s.warp_parts[0][w]), rest = max(rest, s.warp_parts[1][w]);
                st_remote(remote(&s.ranks[rank].in[round], lane), in), st_remote(remote(&s.ranks[rank].rest[round], lane), rest);
            }
            cluster_sync_all();
            in = rest = 0;
            for (int q = 0; q < size; ++q) in = max(in, s.ranks[q].in[round]), rest = max(rest, s.ranks[q].rest[round]);
        };
        u64 own = 0, in = 0, rest = 0;
        if (unit >= 0) {
            float x[kPer], noise[kPer], at = -INFINITY;
            read_scored(unit, x, noise);
#pragma unroll
            for (int j = kPer - 1; j >= 0; --j)  // the first of the unit's tokens with that score
                if (x[j] > -INFINITY && __fadd_rn(-row.t_of(x[j]), noise[j]) == most) own = key_of(most, base + unit * kPer + j), at = x[j];
            float t;
            in = place(at, t) == 0 ? own : 0;
            rest = in ? 0 : own;
        }
        const bool out = rest > 0;
        exchange(0, in, rest);
        if (rest > in && d > 0 && in > 0) {
            u64 more = 0;
            rest = 0;
            if (out && own > in)
                each_scored([&](int i, const float (&x)[kPer], const float (&noise)[kPer]) {
                    if (!(largest(x) >= reach)) return;
                    const float least = value_of(static_cast<uint32_t>(in >> 32));
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        if (!(__fadd_rn(-row.t_of(x[j]), noise[j]) >= least) || x[j] == -INFINITY) continue;
                        float t;
                        const int where = place(x[j], t);
                        const u64 key = key_of(__fadd_rn(-t, noise[j]), base + i * kPer + j);
                        if (where == 0) more = max(more, key);
                        if (where == 1) rest = max(rest, key);
                    }
                });
            exchange(1, more, rest);
            in = max(in, more);
        }
        best = in;
        if (in > rest) {
            if (rank == 0 && tid == 0) answer();
            return;
        }
        // A token of bin d may be drawn: the bin's tokens are packed and ordered.  Without a draw before it (all of
        // them -inf, or NaN, which counts as -inf) the tokens before it are offered one by one.
        const float slack = fabsf(row.top) * 1e-6f + (bins.width * temp) * 1e-2f + range * temp * 1e-6f;
        float edge = row.top - (d + 0.5f) * bins.width * temp - slack;  // below any token of bin d
        if (!(edge > reach && d < kBins - 1 && plain && row.top < INFINITY)) edge = reach;
        float sure = row.top - (d - 0.5f) * bins.width * temp + slack;  // above any
        if (!(edge > reach && in > 0)) sure = INFINITY;
        each_unit([&](int i, const float (&x)[kPer]) {
            if (!(largest(x) >= edge)) return;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (!(x[j] >= edge && x[j] > -INFINITY && !(x[j] > sure))) continue;
                if (in > 0) {
                    keep(x[j], base + i * kPer + j);  // of bin d or beside it
                } else {
                    const float t = row.t_of(x[j]);
                    const int b = bins.bin(t), token = base + i * kPer + j;
                    if (b == d) keep(x[j], token);
                    else if (b < d && (low == 0.f || expf(-t) >= low)) offer(t, noise_of(e0 + token), token);
                }
            }
        });
        __syncthreads();
        tokens = static_cast<int>(s.maybe_n);
        reach = edge;
        cluster_sync_all();  // nobody reads the bins any more
        histogram(bins, level0, ~0ull);
        cluster_sync_all();
        const Scan all = totals(bins, level0, each);
        if (tid == d) s.here = all.count;
        __syncthreads();
        u64 kept;
        threshold = refine(bins, d, true, need_here, s.here, each, ~0ull, false, &kept);
    }
    each_token([&](float v, int i) {
        const float t = row.t_of(v);
        if (order_of(v, i) <= threshold && (low == 0.f || expf(-t) >= low)) offer(t, noise_of(e0 + i), i);
    });
    __syncthreads();
    answer_of_all();
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    cluster_arrive_release();  // waited for before the first access to another CTA's shared memory
    pdl_trigger_and_wait();
    Sampler<kF32> sampler(*reinterpret_cast<Shared *>(smem), smem + sizeof(Shared), a);
    sampler.run(sampler.row_of(blockIdx.x / cluster_size()));
}

template <bool kF32>
cudaError_t launch_typed(SampleArgs &a, const DevCtx &ctx, cudaStream_t stream) {
    constexpr int kPer = kF32 ? 4 : 8;
    // The largest cluster of which the resident CTAs hold all rows at once, or twice that number where rows may take
    // top-p, which takes longer; and slices of 2048 logits at least.  256 rows of 128256 fp32 logits in clusters of 1, 2, 4:
    // every kind 113, 75, 91 us (the same logits), but unfiltered 58, 67, 80, top-k 65, 68, 89, min-p 36, 41, 53, greedy
    // 31, 37, 47.  Whether a top_p is given decides, not its values, which the host has not: all ones take as long.
    const int64_t ctas = (a.top_p ? 2 : 1) * kCtasPerSm * ctx.num_sms;
    int size = 1;
    while (size < kMaxCluster && a.m * size * 2 <= ctas && a.vocab > size * 4096) size *= 2;
    const int units = a.vocab % kPer ? (a.vocab + 2 * kPer - 2) / kPer : a.vocab / kPer;  // what a row touches, at worst
    a.slice_units = (units + size - 1) / size;
    a.parts = std::min(65535.f, std::floor(4294960000.f / static_cast<float>(a.slice_units * kPer)));
    // room for as many tokens as lets all the CTAs that the registers allow share an SM
    const int room = (226 * 1024 / kCtasPerSm - 1024 - static_cast<int>(sizeof(Shared))) / 8 / 16 * 16;
    a.most = std::min((a.slice_units * kPer + 15) / 16 * 16, room);
    constexpr auto kernel = sample_kernel<kF32>;
    const cudaError_t e = allow_smem<kernel>(227 * 1024, ctx.device);
    if (e != cudaSuccess) return e;
    // in more than one wave, and while looking through all rows takes less time than a row
    a.sorted = a.top_p != nullptr && a.m * size > kCtasPerSm * ctx.num_sms && a.m <= 4096;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.m * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + static_cast<size_t>(a.most) * 8;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_sample(const void *logits, int32_t logits_type, int64_t m, int64_t vocab, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, const float *noise,
                          int32_t *ids, float *logprob, const DevCtx &ctx, cudaStream_t stream) {
    SampleArgs a;
    a.logits = static_cast<const uint8_t *>(logits);
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.noise = noise;
    a.ids = ids;
    a.logprob = logprob;
    a.status = ctx.status;
    a.m = m;
    a.vocab = static_cast<int32_t>(vocab);
    const bool f32 = logits_type == BD_LOGITS_F32;
    return f32 ? launch_typed<true>(a, ctx, stream) : launch_typed<false>(a, ctx, stream);
}

}  // namespace bd
