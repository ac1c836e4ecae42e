// sample.cu -- draw of the next token of each row: temperature, top-k, top-p,
// min-p and the Gumbel maximum over what they keep.
//
//   z_i = (x_i - M) / T,  w_i = exp(z_i),  id = argmax over kept of z_i + g_i
//
// Bound: HBM for many rows (the logits once, the noise at kept tokens), latency
// for one.  A row belongs to a cluster of CTAs; each keeps its slice of the
// logits in shared memory, so every pass after the first reads no global
// memory but noise.
//
// The filters are a threshold in the order (x descending, index ascending).
// It is found without sorting: a histogram over t = -z in 2048 bins of 1/64
// holds each bin's count and weight; a scan over the bins finds the one that
// the k-th token or the share p falls into; the few tokens of that bin (or,
// where all tokens up to it are few, all of them) are gathered and ordered
// exactly.  A bin with too many tokens is split again, first by the remaining
// bits of t, then by the bits of (x, index), which differ for any two tokens.
//
// Sums of weights are integers, so their value does not depend on the order of
// the atomics: within a bin w = exp(-bin / 64) * w' with w' in (63/64, 1], and
// a bin sums round((w' - 63/64) * 2^22) in 32 bits beside its count; across
// bins weights are fixed-point with 40 fractional bits.
#include <algorithm>

#include "bd_device.cuh"
#include "bd_internal.h"

namespace bd {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinBits = 11;
constexpr float kPerUnit = 64.f;  // bins per unit of t; the last bin takes everything from 31.98 on
constexpr int kCap = kThreads;    // tokens ordered exactly, one per thread
constexpr int kIndexBits = 18;    // BD_SAMPLE_MAX_VOCAB = 2^18
constexpr int kMaxCluster = 8;
constexpr int kMaxSmem = 227 * 1024;
constexpr float kFloor = 63.f / 64.f;
constexpr float kFrac = 4194304.f;  // 2^22
constexpr float kFixed = 1099511627776.f;  // 2^40

struct SampleArgs {
    const uint8_t *logits;
    const float *temperature, *top_p, *min_p, *noise;
    const int32_t *top_k;
    int32_t *ids;
    float *logprob;
    unsigned *status;
    int64_t m;
    int32_t vocab, slice_groups;  // groups of 8 logits in a CTA's slice
};

// What the cluster's CTAs have to know of a selection's progress.
struct Choice {
    unsigned long long prefix;
    int depth, bin, sub, shift;
    int list;  // 0: split the bin once more; 1: gather it; 2: gather all bins up to it; 3: no threshold
};

struct alignas(16) Shared {
    uint32_t count[kBins], frac[kBins];  // this CTA's slice
    unsigned long long mass[kBins];      // rank 0: the cluster's totals
    uint32_t total[kBins];
    unsigned long long list_order[kCap], list_mass[kCap];  // rank 0
    unsigned long long scan_mass[kWarps];
    uint32_t scan_count[kWarps];
    unsigned long long best[kMaxCluster];
    unsigned long long threshold;  // keep a token whose order is at most this
    unsigned long long weight_sum;
    float rank_value[2][kMaxCluster], warp_value[kWarps];
    uint32_t list_n;
    int found;
    Choice choice;
};

static_assert(sizeof(Shared) % 16 == 0, "the slice of logits behind it is stored in 16-byte pieces");

// ---- cluster shared memory ----------------------------------------------------------
__device__ __forceinline__ void cluster_sync_all() {
    __syncthreads();  // the barrier's instructions want converged warps
    cluster_arrive_release();
    cluster_wait_acquire();
}
__device__ __forceinline__ uint32_t remote(const void *p, int rank) { return mapa_rank(smem_u32(p), rank); }
__device__ __forceinline__ void st_remote32(uint32_t at, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void st_remote64(uint32_t at, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_remote32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t add_remote32(uint32_t at, uint32_t v) {
    uint32_t old;
    asm volatile("atom.add.shared::cluster.u32 %0, [%1], %2;" : "=r"(old) : "r"(at), "r"(v) : "memory");
    return old;
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
// Bits that ascend with the value (no NaN, no -0).
__device__ __forceinline__ uint32_t ascending(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
// Smaller = earlier: larger logit first, then lower index.
__device__ __forceinline__ unsigned long long order_of(float x, int i) {
    return static_cast<unsigned long long>(~ascending(x)) << kIndexBits | static_cast<unsigned>(i);
}
struct Row {
    float top, inv_t;
    // -z, at least 0; infinite where the weight is 0
    __device__ __forceinline__ float t_of(float x) const {
        // the largest logit gives 0 also where top or inv_t is infinite
        return x == top ? 0.f : fminf(__fmul_rn(__fsub_rn(top, x), inv_t), INFINITY);
    }
};
__device__ __forceinline__ int bin_of(float t) {
    return t < (kBins - 1) / kPerUnit ? static_cast<int>(t * kPerUnit) : kBins - 1;
}
__device__ __forceinline__ int sub_of(float t, int bin) {
    return bin == kBins - 1 ? 0 : static_cast<int>((t * kPerUnit - bin) * kBins);
}
// round((w' - 63/64) * 2^22); the last bin's weights count as 0 (below 2^-46 of the largest each)
__device__ __forceinline__ uint32_t frac_of(float t, int bin) {
    return bin == kBins - 1 ? 0u : __float2uint_rn((expf(bin * (1.f / kPerUnit) - t) - kFloor) * kFrac);
}
__device__ __forceinline__ unsigned long long mass_of(int bin, uint32_t count, unsigned long long frac) {
    if (bin == kBins - 1) return 0;
    const double w = static_cast<double>(count) * kFloor + static_cast<double>(frac) * (1. / kFrac);
    return static_cast<unsigned long long>(w * (static_cast<double>(expf(bin * (-1.f / kPerUnit))) * kFixed));
}

template <bool kMax>
__device__ __forceinline__ float block_fold(float v, float *smem) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = kMax ? fmaxf(v, u) : v + u;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) smem[threadIdx.x / 32] = v;
    __syncthreads();
    float r = smem[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) r = kMax ? fmaxf(r, smem[w]) : r + smem[w];
    return r;
}
// The same over the cluster, in rank order, in every thread.  A maximum and a sum have a place
// each: one may still be read while a faster CTA writes the other.
template <bool kMax>
__device__ __forceinline__ float cluster_fold(float v, Shared &s, int rank, int size) {
    v = block_fold<kMax>(v, s.warp_value);
    if (threadIdx.x < size) st_remote32(remote(&s.rank_value[kMax][rank], threadIdx.x), __float_as_uint(v));
    cluster_sync_all();
    float r = s.rank_value[kMax][0];
    for (int c = 1; c < size; ++c) r = kMax ? fmaxf(r, s.rank_value[kMax][c]) : r + s.rank_value[kMax][c];
    return r;
}

// One slice of logits in shared memory: element e of the slice is the row's token base + e.
template <bool kF32>
struct Slice {
    const uint8_t *data;
    int base, groups;
    __device__ __forceinline__ float at(int e) const {
        if constexpr (kF32) return reinterpret_cast<const float *>(data)[e];
        return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(data)[e]) << 16);
    }
};

// Finds the threshold of one filter among tokens whose order is at most `limit`: the first k
// tokens (by_mass false) or the shortest prefix of weight p (by_mass true).  With joint_p < 1 and
// few tokens up to the k-th, the share p is taken in the same step (*joint_done).
template <bool kF32>
__device__ void select(const Slice<kF32> &sl, const Row &row, Shared &s, int rank, int size, bool by_mass,
                       unsigned long long limit, uint32_t k, float p, float joint_p, bool *joint_done,
                       unsigned long long *all_mass) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    Choice at = {0, 0, 0, 0, 0, 0};
    unsigned long long need = k;  // rank 0: count or weight still to cover
    while (true) {
        // this CTA's histogram at the current depth
        for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0, s.frac[i] = 0;
        __syncthreads();
        for (int e = tid; e < sl.groups * 8; e += kThreads) {
            const float x = sl.at(e);
            if (x == -INFINITY) continue;
            const unsigned long long o = order_of(x, sl.base + e);
            if (o > limit) continue;
            const float t = row.t_of(x);
            const int bin = bin_of(t);
            int digit = bin;
            if (at.depth > 0) {
                if (bin != at.bin) continue;
                digit = sub_of(t, bin);
                if (at.depth > 1) {
                    if (digit != at.sub || (at.depth > 2 && o >> (at.shift + kBinBits) != at.prefix)) continue;
                    digit = static_cast<int>(o >> at.shift) & (kBins - 1);
                }
            }
            atomicAdd(&s.count[digit], 1u);
            atomicAdd(&s.frac[digit], frac_of(t, bin));
        }
        cluster_sync_all();
        // totals of a share of the bins each, left with rank 0
        const int share = kBins / size;
        for (int i = tid; i < share; i += kThreads) {
            const int d = rank * share + i;
            uint32_t n = 0;
            unsigned long long f = 0;
            for (int c = 0; c < size; ++c) {
                n += ld_remote32(remote(&s.count[d], c));
                f += ld_remote32(remote(&s.frac[d], c));
            }
            st_remote32(remote(&s.total[d], 0), n);
            st_remote64(remote(&s.mass[d], 0), mass_of(at.depth == 0 ? d : at.bin, n, f));
        }
        cluster_sync_all();
        if (rank == 0) {
            // inclusive scan over the bins, four per thread
            constexpr int kPer = kBins / kThreads;
            uint32_t n[kPer], n_sum = 0;
            unsigned long long w[kPer], w_sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                n_sum += s.total[tid * kPer + i], w_sum += s.mass[tid * kPer + i];
                n[i] = n_sum, w[i] = w_sum;
            }
            uint32_t n_in = n_sum;
            unsigned long long w_in = w_sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t a = __shfl_up_sync(0xFFFFFFFFu, n_in, o);
                const unsigned long long b = __shfl_up_sync(0xFFFFFFFFu, w_in, o);
                if (lane >= o) n_in += a, w_in += b;
            }
            if (lane == 31) s.scan_count[warp] = n_in, s.scan_mass[warp] = w_in;
            if (tid == 0) s.found = kBins, s.list_n = 0;
            __syncthreads();
            uint32_t n_before = n_in - n_sum, n_all = 0;
            unsigned long long w_before = w_in - w_sum, w_all = 0;
            for (int i = 0; i < kWarps; ++i) {
                if (i < warp) n_before += s.scan_count[i], w_before += s.scan_mass[i];
                n_all += s.scan_count[i], w_all += s.scan_mass[i];
            }
            if (at.depth == 0) {
                *all_mass = w_all;
                if (by_mass) need = static_cast<unsigned long long>(static_cast<double>(p) * static_cast<double>(w_all));
                if (by_mass && need == 0) need = 1;  // the first token always stays
            }
            // the first bin that reaches what is needed; the last non-empty one if rounding keeps all short of it
            int mine = kBins, last = -1;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i) {
                if ((by_mass ? w_before + w[i] : n_before + n[i]) >= need) mine = tid * kPer + i;
                if (last < 0 && n[i] > (i ? n[i - 1] : 0)) last = tid * kPer + i;
            }
            if (mine < kBins) atomicMin(&s.found, mine);
            __syncthreads();
            const bool reached = s.found < kBins;
            __syncthreads();
            if (!reached) {
                if (tid == 0) s.found = -1;
                __syncthreads();
                if (last >= 0) atomicMax(&s.found, last);
                __syncthreads();
            }
            const int d = s.found;
            if (d / kPer == tid) {
                const int i = d % kPer;
                uint32_t nb = n_before;
                unsigned long long wb = w_before;
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (q < i) nb = n_before + n[q], wb = w_before + w[q];
                const uint32_t here = s.total[d];
                Choice c = at;
                if (at.depth == 0) c.bin = d;
                else if (at.depth == 1) c.sub = d;
                else c.prefix = at.prefix << kBinBits | static_cast<unsigned>(d);
                if (!reached && at.depth == 0) {
                    c.list = 3;  // fewer tokens than k, or all of them for the share p
                } else if (!by_mass && at.depth == 0 && joint_p < 1.f && nb + here <= kCap) {
                    c.list = 2;
                } else {
                    need -= by_mass ? wb : nb;
                    c.list = here <= kCap;
                    // the next level's digit: 50 bits of order from the top, 11 at a time
                    c.depth = at.depth + 1;
                    if (c.depth == 2) c.shift = 32 + kIndexBits - kBinBits, c.prefix = 0;
                    if (c.depth > 2) c.shift = at.shift - kBinBits;
                    if (c.shift < 0) c.list = 1;  // all bits used: one token
                }
                s.scan_mass[0] = need;
                for (int r = 0; r < size; ++r) {
                    const uint32_t to = remote(&s.choice, r);
                    st_remote64(to, c.prefix);
                    st_remote32(to + 8, c.depth), st_remote32(to + 12, c.bin), st_remote32(to + 16, c.sub);
                    st_remote32(to + 20, c.shift), st_remote32(to + 24, c.list);
                }
            }
            __syncthreads();
            need = s.scan_mass[0];
        }
        cluster_sync_all();
        const int depth = at.depth;
        at = s.choice;
        if (at.list == 0) continue;
        if (at.list == 3) {
            if (tid == 0) s.threshold = limit;
            __syncthreads();
            return;
        }
        // gather the bin (or the bins up to it) with rank 0
        for (int e = tid; e < sl.groups * 8; e += kThreads) {
            const float x = sl.at(e);
            if (x == -INFINITY) continue;
            const unsigned long long o = order_of(x, sl.base + e);
            if (o > limit) continue;
            const float t = row.t_of(x);
            const int bin = bin_of(t);
            if (at.list == 2 ? bin > at.bin : bin != at.bin) continue;
            if (depth > 0 && sub_of(t, bin) != at.sub) continue;
            if (depth > 1) {
                const int shift = at.shift + kBinBits;
                if (o >> shift != at.prefix) continue;
            }
            const uint32_t slot = add_remote32(remote(&s.list_n, 0), 1u);
            if (slot < kCap) {
                st_remote64(remote(&s.list_order[slot], 0), o);
                st_remote64(remote(&s.list_mass[slot], 0), mass_of(bin, 1, frac_of(t, bin)));
            }
        }
        cluster_sync_all();
        if (rank == 0) {
            const int n = min(s.list_n, static_cast<uint32_t>(kCap));
            const bool on = tid < n;
            const unsigned long long o = on ? s.list_order[tid] : ~0ull;
            uint32_t before = 0;
            unsigned long long w_before = 0, w_kept = 0;
            for (int j = 0; j < n; ++j) {
                const bool earlier = s.list_order[j] < o;
                before += earlier;
                w_before += earlier ? s.list_mass[j] : 0;
            }
            bool keep = on && (by_mass ? w_before < need : before < need);
            if (tid == 0) s.threshold = 0, s.weight_sum = 0;
            __syncthreads();
            if (at.list == 2) {
                if (keep) atomicAdd(&s.weight_sum, s.list_mass[tid]);
                __syncthreads();
                w_kept = s.weight_sum;
                const double target = static_cast<double>(joint_p) * static_cast<double>(w_kept);
                keep = keep && (before == 0 || static_cast<double>(w_before) < target);
            }
            if (keep) atomicMax(&s.threshold, o);
            __syncthreads();
            if (tid > 0 && tid < size) st_remote64(remote(&s.threshold, tid), s.threshold);
        }
        cluster_sync_all();
        *joint_done = at.list == 2;
        return;
    }
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    uint8_t *data = smem + sizeof(Shared);
    cluster_arrive_release();  // waited for before the first access to another CTA's shared memory
    pdl_trigger_and_wait();
    const int tid = threadIdx.x, rank = cluster_rank(), size = cluster_size();
    const int64_t r = blockIdx.x / size;
    // groups of 8 logits at multiples of 8 of the whole array: 16-byte aligned in both types, noise included
    const int64_t e0 = r * a.vocab, e1 = e0 + a.vocab;
    const int64_t g0 = e0 / 8 + static_cast<int64_t>(rank) * a.slice_groups;
    const int64_t g1 = min(g0 + a.slice_groups, (e1 + 7) / 8);
    Slice<kF32> sl;
    sl.data = data;
    sl.groups = g1 > g0 ? static_cast<int>(g1 - g0) : 0;
    sl.base = static_cast<int>(g0 * 8 - e0);
    float top = -INFINITY;
    for (int g = tid; g < sl.groups; g += kThreads) {
        const int64_t e = (g0 + g) * 8;
        float x[8];
        if (e >= e0 && e + 8 <= e1) {
            if constexpr (kF32) {
                const uint4 u = ldg_stream(a.logits + e * 4), v = ldg_stream(a.logits + e * 4 + 16);
                x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z);
                x[3] = __uint_as_float(u.w), x[4] = __uint_as_float(v.x), x[5] = __uint_as_float(v.y);
                x[6] = __uint_as_float(v.z), x[7] = __uint_as_float(v.w);
            } else {
                const uint4 u = ldg_stream(a.logits + e * 2);
                x[0] = bf16lo_to_f32(u.x), x[1] = bf16hi_to_f32(u.x), x[2] = bf16lo_to_f32(u.y);
                x[3] = bf16hi_to_f32(u.y), x[4] = bf16lo_to_f32(u.z), x[5] = bf16hi_to_f32(u.z);
                x[6] = bf16lo_to_f32(u.w), x[7] = bf16hi_to_f32(u.w);
            }
        } else {  // the row's ragged ends, element by element
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = -INFINITY;
                if (e + j >= e0 && e + j < e1) {
                    if constexpr (kF32) x[j] = reinterpret_cast<const float *>(a.logits)[e + j];
                    else x[j] = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(a.logits)[e + j]) << 16);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = fmaxf(x[j], -INFINITY) + 0.f;  // NaN to -inf, -0 to +0
            top = fmaxf(top, x[j]);
        }
        uint4 *d = reinterpret_cast<uint4 *>(data);
        if constexpr (kF32) {
            d[2 * g] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            d[2 * g + 1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
        } else {
            d[g] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        }
    }
    __syncthreads();
    cluster_wait_acquire();
    Row row;
    row.top = cluster_fold<true>(top, s, rank, size);
    const float temp = a.temperature ? a.temperature[r] : 1.f;
    const bool greedy = !(temp > 0.f);
    row.inv_t = greedy ? 1.f : __fdiv_rn(1.f, temp);
    const int top_k = a.top_k ? a.top_k[r] : 0;
    uint32_t k = top_k > 0 && top_k < a.vocab ? static_cast<uint32_t>(top_k) : 0;
    float p = a.top_p ? a.top_p[r] : 1.f;
    if (p <= 0.f) k = 1;
    if (!(p > 0.f && p < 1.f) || k == 1) p = 1.f;
    float low = a.min_p ? a.min_p[r] : 0.f;
    low = low > 0.f ? fminf(low, 1.f) : 0.f;

    unsigned long long threshold = ~0ull, all_mass = 0;
    const bool filtered = !greedy && (k > 0 || p < 1.f) && row.top > -INFINITY;
    if (filtered) {
        bool done = false;
        if (k > 0) {
            select(sl, row, s, rank, size, false, threshold, k, 1.f, p, &done, &all_mass);
            threshold = s.threshold;
        }
        if (p < 1.f && !done) {
            unsigned long long mass = 0;
            cluster_sync_all();  // s.threshold is read above before it is written again
            select(sl, row, s, rank, size, true, threshold, 0, p, 1.f, &done, &mass);
            if (k == 0) all_mass = mass;
            threshold = s.threshold;
        }
    }

    // the kept token of the largest score, and for a row without a histogram the sum of all weights
    unsigned long long best = 0;
    float sum = 0.f;
    for (int e = tid; e < sl.groups * 8; e += kThreads) {
        const float x = sl.at(e);
        if (x == -INFINITY) continue;
        const float t = row.t_of(x);
        const float w = expf(-t);
        if (!filtered) sum += w;
        if (order_of(x, sl.base + e) > threshold || w < low) continue;
        float score = -t;
        if (!greedy) score = __fadd_rn(score, fmaxf(a.noise[e0 + sl.base + e], -INFINITY));
        const unsigned long long c =
            static_cast<unsigned long long>(ascending(fmaxf(score, -INFINITY) + 0.f)) << 32 | (0xFFFFFFFFu - static_cast<unsigned>(sl.base + e));
        best = c > best ? c : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const unsigned long long u = __shfl_xor_sync(0xFFFFFFFFu, best, o);
        best = u > best ? u : best;
    }
    __syncthreads();
    if (tid % 32 == 0) s.scan_mass[tid / 32] = best;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) best = s.scan_mass[w] > best ? s.scan_mass[w] : best;
        st_remote64(remote(&s.best[rank], 0), best);
    }
    sum = cluster_fold<false>(sum, s, rank, size);
    if (rank == 0 && tid == 0) {
        for (int c = 0; c < size; ++c) best = s.best[c] > best ? s.best[c] : best;
        const int id = best ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
        a.ids[r] = id;
        if (a.logprob) {
            float lp = -INFINITY;
            if (id >= 0) {
                float x;
                if constexpr (kF32) x = reinterpret_cast<const float *>(a.logits)[e0 + id];
                else x = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(a.logits)[e0 + id]) << 16);
                if (filtered) sum = static_cast<float>(static_cast<double>(all_mass) / kFixed);
                lp = -row.t_of(x) - logf(sum);
            }
            a.logprob[r] = lp;
        }
    }
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
    // a slice of about 16384 logits per CTA
    int size = 1;
    while (size < kMaxCluster && vocab > size * int64_t{16384}) size *= 2;
    const int64_t groups = vocab / 8 + 2;  // an unaligned row touches up to this many groups
    a.slice_groups = static_cast<int32_t>((groups + size - 1) / size);
    const size_t smem = sizeof(Shared) + static_cast<size_t>(a.slice_groups) * 8 * (f32 ? 4 : 2);
    auto kernel = f32 ? sample_kernel<true> : sample_kernel<false>;
    const cudaError_t e = f32 ? allow_smem<sample_kernel<true>>(kMaxSmem, ctx.device)
                              : allow_smem<sample_kernel<false>>(kMaxSmem, ctx.device);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(m * size));
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
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace bd
