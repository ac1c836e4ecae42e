// sample.cu -- draw of the next token of each row: temperature, top-k, top-p,
// min-p and the Gumbel maximum over what they keep.
//
//   z_i = (x_i - M) / T,  w_i = exp(z_i),  id = argmax over kept of z_i + g_i
//
// Bound: HBM for many rows (the logits once, the noise at kept tokens), latency
// for one.  A row belongs to a cluster of CTAs, each with a slice of it in shared
// memory, so global memory is read once but for noise.  The passes are short
// loops: the same steps unrolled over registers were bound by fetching their code.
//
// The filters are a threshold in the order (x descending, index ascending), found
// without sorting:
//  1. Tokens that cannot be kept are left out.  top-k: every warp of the cluster has
//     j = ceil(k / warps) threads whose largest logit reaches the warp's j-th largest, so
//     k tokens reach the smallest of these.  top-p: tokens with t = -z above
//     ln(V / ((1 - p) sum w)) weigh less than (1 - p) sum w together, so the prefix
//     ends before them.
//  2. A histogram over t, one bin per thread, holds each bin's count and weight.  Every
//     CTA adds up the cluster's bins and scans them, and finds the bin that the k-th
//     token or the share p falls into.
//  3. The tokens of that bin (all bins up to it, if those are few: top-k as used) are
//     sent to every CTA and ordered exactly.  A bin with too many tokens is split again,
//     by the remaining bits of t, then by the bits of (x, index), which differ for any two.
//
// Sums of weights do not depend on the order of atomics: within a bin of width d,
// w = exp(-bin d) w' with w' in [1 - d, 1], and a bin sums round((w' - 1 + d) 65535 / d)
// in 32 bits beside its count; across bins weights are fixed-point with 40 fractional
// bits.  The sum of all weights is fp32 in an order fixed by the shape.
#include <algorithm>

#include "bd_device.cuh"
#include "bd_internal.h"

namespace bd {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;
constexpr int kBits = 9;            // a digit: one bin
constexpr int kCap = 256;           // tokens ordered exactly
constexpr int kMaybe = 2048;        // places of tokens that may be kept; with more of them passes go over the slice
constexpr int kIndexBits = 18;      // BD_SAMPLE_MAX_VOCAB = 2^18
constexpr int kMaxCluster = 8;
constexpr int kMaxSmem = 160 * 1024;  // a slice of 32768 fp32 logits and the rest
constexpr float kRange = 31.5f;     // weights below exp(-31.5) of the largest count as 0 in a prefix's sum
constexpr float kFixed = 1099511627776.f;  // 2^40
constexpr float kLog2e = 1.44269504088896f;

using u64 = unsigned long long;

struct SampleArgs {
    const uint8_t *logits;
    const float *temperature, *top_p, *min_p, *noise;
    const int32_t *top_k;
    int32_t *ids;
    float *logprob;
    int64_t m;
    int32_t vocab, slice_units;  // 16-byte units of logits in a CTA's slice
};

struct alignas(16) Shared {
    uint2 bins[kBins];  // count, weight
    u64 list_order[kCap], list_mass[kCap], sorted_mass[kCap];
    uint16_t maybe[kMaybe];
    u64 warp_mass[kWarps], warp_parts[2][kWarps];
    uint32_t warp_count[kWarps];
    float warp_value[3][kWarps];
    // written by the cluster's CTAs
    float rank_top[kMaxCluster], rank_sum[kMaxCluster], rank_low[kMaxCluster];
    u64 rank_best[kMaxCluster];
    // written by one thread for its CTA
    u64 before_mass, kept_mass, threshold;
    uint32_t before_count, here, list_n, maybe_n;
    int found;
};
static_assert(sizeof(Shared) % 16 == 0, "the slice of logits behind it is stored in 16-byte units");

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
__device__ __forceinline__ uint2 ld_remote(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
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
// Bits that ascend with the value (no NaN, no -0), and back.
__device__ __forceinline__ uint32_t ascending(float f) {
    const uint32_t u = __float_as_uint(f);
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
// Bins of equal width over [0, range); the last one takes everything from `range` on and weighs nothing.
struct Bins {
    float scale, width, unit;  // 1 / width, width, 65535 / width
    __device__ __forceinline__ explicit Bins(float range)
        : scale((kBins - 1) / range), width(range / (kBins - 1)), unit(65535.f * scale) {}
    __device__ __forceinline__ int bin(float t) const {
        return t < width * (kBins - 1) ? min(static_cast<int>(t * scale), kBins - 2) : kBins - 1;
    }
    __device__ __forceinline__ int sub(float t, int b) const {  // the same again within a bin
        return b == kBins - 1 ? 0 : min(max(static_cast<int>((t * scale - b) * kBins), 0), kBins - 1);
    }
    __device__ __forceinline__ uint32_t part(float t, int b) const {
        return b == kBins - 1 ? 0u : __float2uint_rn(fmaxf(ex2((b * width - t) * kLog2e) - (1.f - width), 0.f) * unit);
    }
    // fp32 from whole numbers: the same on every CTA, 2^-22 of the weight
    __device__ __forceinline__ u64 mass(int b, uint32_t count, u64 parts) const {
        if (b == kBins - 1) return 0;
        const float w = fmaf(static_cast<float>(parts), width * (1.f / 65535.f), static_cast<float>(count) * (1.f - width));
        return __float2ull_rn(w * (ex2(b * width * -kLog2e) * kFixed));
    }
};
// floor(p * mass) for 0 < p < 1, at least 1: the first token always stays
__device__ __forceinline__ u64 share_of(float p, u64 mass) {
    return max(__umul64hi(__float2ull_rz(p * 18446744073709551616.f), mass), u64{1});
}

template <bool kF32>
struct Sampler {
    static constexpr int kPer = kF32 ? 4 : 8;  // logits of a unit

    Shared &s;
    const SampleArgs &a;
    uint8_t *slice;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, rank = cluster_rank(), size = cluster_size();
    int base = 0, units = 0;  // token of the slice's first element, units in the slice
    int tokens = 0;           // how many tokens the passes of a filter go over
    bool some = false;        // ... those in s.maybe, or all of the slice
    float reach = -INFINITY;  // tokens below it are not kept
    Row row;

    __device__ Sampler(Shared &shared, uint8_t *data, const SampleArgs &args) : s(shared), a(args), slice(data) {}

    __device__ __forceinline__ float at(int e) const {
        if constexpr (kF32) return reinterpret_cast<const float *>(slice)[e];
        return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(slice)[e]) << 16);
    }
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[kPer]) {
        if constexpr (kF32) {
            x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
        } else {
            x[0] = bf16lo_to_f32(u.x), x[1] = bf16hi_to_f32(u.x), x[2] = bf16lo_to_f32(u.y), x[3] = bf16hi_to_f32(u.y);
            x[4] = bf16lo_to_f32(u.z), x[5] = bf16hi_to_f32(u.z), x[6] = bf16lo_to_f32(u.w), x[7] = bf16hi_to_f32(u.w);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[kPer]) {
        if constexpr (kF32)
            return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        else
            return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    // f(x, token) for this thread's share of the tokens that may be kept
    template <class F>
    __device__ __forceinline__ void each_token(F f) const {
        for (int i = tid; i < tokens; i += kThreads) {
            const int e = some ? s.maybe[i] : i;
            const float x = at(e);
            if (x >= reach && x > -INFINITY) f(x, base + e);
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

    // Counts and weights of the bins up to each thread's one.
    struct Scan {
        uint32_t count, count_upto, count_all;
        u64 mass, mass_upto, mass_all;
    };
    __device__ __forceinline__ Scan scan(uint32_t count, u64 mass) {
        Scan r = {count, count, 0, mass, mass, 0};
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, r.count_upto, o);
            const u64 w = __shfl_up_sync(0xFFFFFFFFu, r.mass_upto, o);
            if (lane >= o) r.count_upto += n, r.mass_upto += w;
        }
        __syncthreads();
        if (lane == 31) s.warp_count[warp] = r.count_upto, s.warp_mass[warp] = r.mass_upto;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t n = s.warp_count[w];
            const u64 m = s.warp_mass[w];
            if (w < warp) r.count_upto += n, r.mass_upto += m;
            r.count_all += n, r.mass_all += m;
        }
        return r;
    }
    // The first bin at which the count or the weight reaches `need`, what precedes it in s.before_*, its own
    // count in s.here.  Where rounding leaves the sum of all bins short, the last bin that holds a token.
    __device__ __forceinline__ int find(const Scan &c, bool by_mass, u64 need) {
        const u64 all = by_mass ? c.mass_all : c.count_all;
        bool here;
        if (all >= need) {
            here = by_mass ? c.mass_upto >= need && c.mass_upto - c.mass < need : c.count_upto >= need && c.count_upto - c.count < need;
        } else {
            here = c.count > 0 && c.count_upto == c.count_all;
        }
        __syncthreads();
        if (here) s.found = tid, s.before_count = c.count_upto - c.count, s.before_mass = c.mass_upto - c.mass, s.here = c.count;
        __syncthreads();
        return s.found;
    }

    // This CTA's tokens with order <= limit in the set chosen so far, one histogram digit each.
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
    __device__ void histogram(const Bins &bins, const Level &at, u64 limit) {
        s.bins[tid] = make_uint2(0, 0);
        __syncthreads();
        each_token([&](float x, int i) {
            const float t = row.t_of(x);
            const u64 o = order_of(x, i);
            if (o > limit) return;
            const int d = digit_of(bins, at, t, o);
            if (d < 0) return;
            atomicAdd(&s.bins[d].x, 1u);
            atomicAdd(&s.bins[d].y, bins.part(t, at.depth == 0 ? d : at.bin));
        });
    }
    // The cluster's totals of this thread's bin, and the count of each CTA (four 16-bit fields a word).
    __device__ Scan totals(const Bins &bins, const Level &at, u64 (&each)[2]) {
        uint2 v[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) v[c] = c < size ? ld_remote(remote(&s.bins[tid], c)) : make_uint2(0, 0);
        uint32_t n = 0;
        u64 parts = 0;
        each[0] = each[1] = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            n += v[c].x, parts += v[c].y;
            each[c / 4] |= static_cast<u64>(v[c].x) << 16 * (c % 4);
        }
        return scan(n, bins.mass(at.depth == 0 ? tid : at.bin, n, parts));
    }
    // Sends this CTA's tokens of one set to every CTA's list.  `upto`: all bins up to at.bin, else the set of
    // digit d at level `at`.  The places follow from the counts that every CTA has of every other.
    __device__ void gather(const Bins &bins, const Level &at, int d, bool upto, u64 limit, const u64 (&each)[2]) {
        const bool mine = upto ? tid <= d : tid == d;
        u64 e0 = mine ? each[0] : 0, e1 = mine ? each[1] : 0;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) e0 += __shfl_xor_sync(0xFFFFFFFFu, e0, o), e1 += __shfl_xor_sync(0xFFFFFFFFu, e1, o);
        if (lane == 0) s.warp_parts[0][warp] = e0, s.warp_parts[1][warp] = e1;
        if (tid == 0) s.list_n = 0;
        __syncthreads();
        e0 = e1 = 0;
        for (int w = 0; w < kWarps; ++w) e0 += s.warp_parts[0][w], e1 += s.warp_parts[1][w];
        uint32_t first = 0;
        for (int c = 0; c < rank; ++c) first += static_cast<uint32_t>((c < 4 ? e0 : e1) >> 16 * (c % 4)) & 0xFFFFu;
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
        if (tid >= n && tid < kCap) s.list_order[tid] = ~0ull, s.list_mass[tid] = 0;
        __syncthreads();
        // rank by counting, two threads a token, each over half of the list
        const int i = tid / 2, half = tid % 2;
        const u64 mine = s.list_order[i];
        uint32_t before = 0;
        const uint32_t end = (n + 1) / 2;  // pairs
        for (uint32_t j = half; j < end; j += 2) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&s.list_order[2 * j]);
            before += (two.x < mine) + (two.y < mine);
        }
        before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
        if (half == 0 && i < n) s.sorted_mass[before] = s.list_mass[i];
        __syncthreads();
        // weights in that order, one thread a place
        const u64 w = tid < n ? s.sorted_mass[tid] : 0;
        const Scan c = scan(tid < n, w);
        const u64 lighter = c.mass_upto - w;
        bool keep = tid < n && (by_mass ? lighter < need : static_cast<u64>(tid) < need);
        if (share < 1.f) {
            const int last = static_cast<int>(min(need, static_cast<u64>(n))) - 1;
            if (tid == last) s.kept_mass = c.mass_upto;
            __syncthreads();
            keep = keep && lighter < share_of(share, s.kept_mass);
        }
        const int kept = __syncthreads_count(keep);  // they are the first ones
        if (half == 0 && i < n && before == kept - 1) s.threshold = mine;
        if (tid == kept - 1) s.kept_mass = c.mass_upto;
        __syncthreads();
    }

    // The order of the last token to keep of level-0 bin d (`here` tokens, counts by CTA in `each`): its first `need`
    // tokens, or those before which its weight stays below `need`.  `limited`: the bin's counts include tokens
    // beyond `limit`.  *kept receives the weight of the bin's kept tokens.
    __device__ u64 refine(const Bins &bins, int d, bool by_mass, u64 need, uint32_t here, u64 each0, u64 each1, u64 limit, bool limited, u64 *kept) {
        Level at = {0, d, 0, 0, 0};
        u64 each[2] = {each0, each1};
        int digit = d;
        *kept = 0;
        while (here > kCap || limited) {
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

    __device__ void run(int64_t r);
};

template <bool kF32>
__device__ void Sampler<kF32>::run(int64_t r) {
    // units at multiples of kPer of the whole array: 16-byte aligned logits, and 16-byte aligned noise
    const int64_t e0 = r * a.vocab, e1 = e0 + a.vocab;
    const int64_t u0 = e0 / kPer + static_cast<int64_t>(rank) * a.slice_units;
    units = static_cast<int>(max(min(u0 + a.slice_units, (e1 + kPer - 1) / kPer) - u0, int64_t{0}));
    base = static_cast<int>(u0 * kPer - e0);
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

    // the slice, eight loads in flight per thread
    uint4 *data = reinterpret_cast<uint4 *>(slice);
    float top = -INFINITY;
    constexpr int kAtOnce = 8;
    for (int i0 = tid; i0 < units; i0 += kAtOnce * kThreads) {
        uint4 raw[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            const int i = i0 + q * kThreads;
            const int64_t e = (u0 + i) * kPer;
            if (i < units && e >= e0 && e + kPer <= e1) raw[q] = ldg_stream(a.logits + (u0 + i) * 16);
        }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            const int i = i0 + q * kThreads;
            if (i >= units) break;
            const int64_t e = (u0 + i) * kPer;
            float x[kPer];
            if (e >= e0 && e + kPer <= e1) {
                unpack(raw[q], x);
            } else {  // the row's ragged ends, element by element
                for (int j = 0; j < kPer; ++j) {
                    float v = -INFINITY;
                    if (e + j >= e0 && e + j < e1) {
                        if constexpr (kF32) v = reinterpret_cast<const float *>(a.logits)[e + j];
                        else v = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(a.logits)[e + j]) << 16);
                    }
                    if constexpr (kF32) reinterpret_cast<float *>(slice)[i * kPer + j] = v;
                    else reinterpret_cast<uint16_t *>(slice)[i * kPer + j] = static_cast<uint16_t>(__float_as_uint(v) >> 16);
                }
                unpack(data[i], x);
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                x[j] = fmaxf(x[j], -INFINITY) + 0.f;  // NaN to -inf, -0 to +0
                top = fmaxf(top, x[j]);
            }
            data[i] = pack(x);
        }
    }

    // This CTA's largest logit, the sum of its weights relative to it, and for top-k its bound: j threads of every
    // warp reach it.
    if (filtered && k > 0) {
        const uint32_t j = (k + size * kWarps - 1) / (size * kWarps);
        uint32_t left = ascending(top), jth = 0;  // 0: below every logit
        if (j <= 32)
            for (uint32_t i = 0; i < j; ++i) {
                jth = __reduce_max_sync(0xFFFFFFFFu, left);
                const unsigned who = __ballot_sync(0xFFFFFFFFu, left == jth);
                if (lane == __ffs(who) - 1) left = 0;
            }
        reach = jth > ascending(-INFINITY) ? value_of(jth) : -INFINITY;
        if (lane == 0) s.warp_value[0][warp] = reach;
    }
    const float cta_top = block_fold<true>(top, s.warp_value[1]);  // (also: the slice is complete)
    const float per = row.inv_t * kLog2e;
    float sum = 0.f;
    if (cta_top < INFINITY && per > 0.f && per < INFINITY && cta_top > -INFINITY) {
#pragma unroll 2
        for (int i = tid; i < units; i += kThreads) {
            float x[kPer];
            unpack(data[i], x);
#pragma unroll
            for (int j = 0; j < kPer; ++j) sum += ex2((x[j] - cta_top) * per);
        }
    } else if (cta_top > -INFINITY) {  // a logit or a setting at the end of its range
        for (int i = tid; i < units * kPer; i += kThreads) {
            const Row own = {cta_top, row.inv_t};
            if (at(i) > -INFINITY) sum += ex2(own.t_of(at(i)) * -kLog2e);
        }
    }
    sum = block_fold<false>(sum, s.warp_value[2]);
    cluster_wait_acquire();  // every CTA of the cluster runs: its shared memory may be written
    if (tid < size) {
        if (filtered && k > 0)
            for (int w = 0; w < kWarps; ++w) reach = fminf(reach, s.warp_value[0][w]);
        st_remote(remote(&s.rank_top[rank], tid), cta_top);
        st_remote(remote(&s.rank_sum[rank], tid), sum);
        st_remote(remote(&s.rank_low[rank], tid), reach);
    }
    cluster_sync_all();
    row.top = s.rank_top[0];
    for (int c = 1; c < size; ++c) row.top = fmaxf(row.top, s.rank_top[c]);
    if (row.top == -INFINITY) {  // nothing may be drawn; the whole cluster leaves
        if (rank == 0 && tid == 0) {
            a.ids[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        return;
    }
    float weight = 0.f;
    for (int c = 0; c < size; ++c) {
        const float v = s.rank_top[c];
        if (v > -INFINITY) weight = fmaf(s.rank_sum[c], ex2(row.t_of(v) * -kLog2e), weight);
    }

    u64 best = 0;
    auto offer = [&](float t, float noise, int i) {
        float score = -t;
        if (!greedy) score = fmaxf(__fadd_rn(score, fmaxf(noise, -INFINITY)), -INFINITY);
        const u64 c = static_cast<u64>(ascending(score + 0.f)) << 32 | (0xFFFFFFFFu - static_cast<unsigned>(i));
        best = c > best ? c : best;
    };
    auto fold_best = [&] {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) {
            const u64 u = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            best = u > best ? u : best;
        }
        if (lane == 0) s.warp_mass[warp] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) best = s.warp_mass[w] > best ? s.warp_mass[w] : best;
    };
    auto answer = [&] {  // by one thread of the cluster
        const int id = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
        a.ids[r] = id;
        if (a.logprob == nullptr) return;
        float v;
        if constexpr (kF32) v = reinterpret_cast<const float *>(a.logits)[e0 + id];
        else v = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(a.logits)[e0 + id]) << 16);
        a.logprob[r] = -row.t_of(v) - logf(weight);
    };
    auto answer_of_all = [&] {
        fold_best();
        if (tid == 0) st_remote(remote(&s.rank_best[rank], 0), best);
        cluster_sync_all();
        if (rank == 0 && tid == 0) {
            for (int c = 0; c < size; ++c) best = s.rank_best[c] > best ? s.rank_best[c] : best;
            answer();
        }
    };
    if (!filtered) {  // every token, or those of min-p
        constexpr int kBatch = kF32 ? 4 : 2;  // 16 noise values in flight per thread
        for (int i0 = tid; i0 < units; i0 += kBatch * kThreads) {
            float noise[kBatch][kPer];
            bool whole[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int64_t e = (u0 + i0 + q * kThreads) * kPer;
                whole[q] = !greedy && low == 0.f && i0 + q * kThreads < units && e >= e0 && e + kPer <= e1;
#pragma unroll
                for (int j = 0; j < kPer; j += 4) {
                    const float4 v = whole[q] ? *reinterpret_cast<const float4 *>(a.noise + e + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                    noise[q][j] = v.x, noise[q][j + 1] = v.y, noise[q][j + 2] = v.z, noise[q][j + 3] = v.w;
                }
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int i = i0 + q * kThreads;
                if (i >= units) break;
                const int first = base + i * kPer;
                float x[kPer];
                unpack(data[i], x);
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    if (x[j] == -INFINITY) continue;
                    const float t = row.t_of(x[j]);
                    if (low > 0.f && expf(-t) < low) continue;
                    offer(t, greedy || whole[q] ? noise[q][j] : a.noise[e0 + first + j], first + j);
                }
            }
        }
        answer_of_all();
        return;
    }

    // tokens that may be kept: x >= reach, t < range
    float range = kRange;
    bool pruned = false;  // by weight
    if (k > 0) {
        reach = s.rank_low[0];
        for (int c = 1; c < size; ++c) reach = fminf(reach, s.rank_low[c]);
        if (reach > -INFINITY) range = fminf(range, row.t_of(reach) * 1.0001f + 1e-6f);
    } else if (p < 1.f - 1e-5f) {  // a longer prefix is summed over everything, so that it ends by the sum of its own bins
        const float bound = logf(static_cast<float>(a.vocab) / ((1.f - p) * 0.99f * weight));
        if (bound < kRange && row.top < INFINITY && per > 0.f && per < INFINITY) {
            pruned = true;
            range = fmaxf(bound, 1e-3f);
            reach = row.top - range * temp;
            reach -= fabsf(reach) * 1e-6f;
            if (!(reach > -INFINITY)) reach = -INFINITY;
        }
    }
    if (tid == 0) s.maybe_n = 0;
    __syncthreads();
    constexpr int kRound = 32 / kPer;  // units whose tokens are one mask of 32 bits
    for (int i0 = 0; i0 < units; i0 += kRound * kThreads) {
        uint32_t mask = 0;
#pragma unroll
        for (int q = 0; q < kRound; ++q) {
            const int i = i0 + q * kThreads + tid;
            if (i >= units) break;
            float x[kPer];
            unpack(data[i], x);
#pragma unroll
            for (int j = 0; j < kPer; ++j) mask |= (x[j] >= reach ? 1u : 0u) << (q * kPer + j);
        }
        int place = __popc(mask);
        const int n = place;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, place, o);
            if (lane >= o) place += v;
        }
        uint32_t first = 0;
        if (lane == 31 && place > 0) first = atomicAdd(&s.maybe_n, static_cast<uint32_t>(place));
        place += static_cast<int>(__shfl_sync(0xFFFFFFFFu, first, 31)) - n;
        for (; mask && place < kMaybe; mask &= mask - 1) {
            const int bit = __ffs(mask) - 1;
            s.maybe[place++] = static_cast<uint16_t>((i0 + bit / kPer * kThreads + tid) * kPer + bit % kPer);
        }
    }
    __syncthreads();
    some = s.maybe_n <= kMaybe;
    tokens = some ? static_cast<int>(s.maybe_n) : units * kPer;

    const Bins bins(range);
    const Level level0 = {0, 0, 0, 0, 0};
    histogram(bins, level0, ~0ull);
    cluster_sync_all();
    u64 each[2];
    const Scan c = totals(bins, level0, each);
    u64 threshold = ~0ull;
    if (k > 0) {
        const int d = find(c, false, k);
        const uint32_t upto = s.before_count + s.here, need = k - min(s.before_count, k), here = s.here;
        const u64 before_mass = s.before_mass;
        if (upto <= kCap) {  // few enough to finish here: order all of them, take the share p, draw
            gather(bins, level0, d, true, ~0ull, each);
            cluster_sync_all();
            if (rank != 0) return;
            cut(upto, false, k, p);
            if (tid < upto && s.list_order[tid] <= s.threshold) {
                const float v = value_of(~static_cast<uint32_t>(s.list_order[tid] >> kIndexBits));
                const int i = static_cast<int>(s.list_order[tid] & ((1u << kIndexBits) - 1));
                const float t = row.t_of(v);
                if (low == 0.f || expf(-t) >= low) offer(t, a.noise[e0 + i], i);
            }
            __syncthreads();
            fold_best();
            if (tid == 0) answer();
            return;
        }
        u64 kept;
        threshold = refine(bins, d, false, need, here, each[0], each[1], ~0ull, false, &kept);
        if (p < 1.f) {  // the share p of what is kept: it ends in a bin before d, or in what is kept of d
            const u64 target = share_of(p, before_mass + kept);
            cluster_sync_all();  // nobody reads the list any more
            if (target <= before_mass) {
                const int d2 = find(c, true, target);
                threshold = refine(bins, d2, true, target - s.before_mass, s.here, each[0], each[1], ~0ull, false, &kept);
            } else {
                threshold = refine(bins, d, true, target - before_mass, here, each[0], each[1], threshold, true, &kept);
            }
        }
    } else {
        const u64 need = share_of(p, pruned ? __float2ull_rn(weight * kFixed) : c.mass_all);
        const int d = find(c, true, need);
        u64 kept;
        threshold = refine(bins, d, true, need - min(s.before_mass, need - 1), s.here, each[0], each[1], ~0ull, false, &kept);
    }
    each_token([&](float v, int i) {
        const float t = row.t_of(v);
        if (order_of(v, i) <= threshold && (low == 0.f || expf(-t) >= low)) offer(t, a.noise[e0 + i], i);
    });
    answer_of_all();
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    cluster_arrive_release();  // waited for before the first access to another CTA's shared memory
    pdl_trigger_and_wait();
    Sampler<kF32> sampler(*reinterpret_cast<Shared *>(smem), smem + sizeof(Shared), a);
    sampler.run(blockIdx.x / cluster_size());
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
    a.m = m;
    a.vocab = static_cast<int32_t>(vocab);
    const bool f32 = logits_type == BD_LOGITS_F32;
    // slices of about 16384 logits
    int size = 1;
    while (size < kMaxCluster && vocab > size * int64_t{16384}) size *= 2;
    const int per = f32 ? 4 : 8;
    const int64_t units = vocab % per ? (vocab + 2 * per - 2) / per : vocab / per;  // what a row touches, at worst
    a.slice_units = static_cast<int32_t>((units + size - 1) / size);
    const size_t smem = sizeof(Shared) + static_cast<size_t>(a.slice_units) * 16;
    const cudaError_t e = f32 ? allow_smem<sample_kernel<true>>(kMaxSmem, ctx.device)
                              : allow_smem<sample_kernel<false>>(kMaxSmem, ctx.device);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.m * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return f32 ? cudaLaunchKernelEx(&cfg, sample_kernel<true>, a) : cudaLaunchKernelEx(&cfg, sample_kernel<false>, a);
}

}  // namespace bd
