// rotary.cu -- table of rotary positions, scaled for long contexts.
//
//   table[p, i] = amplitude cos(p f_i),  table[p, d + i] = amplitude sin(p f_i)
//
// Bound: HBM (the table is written once).  Angles are whole numbers of 2^-64 turns: a pair's turns per position, as such a
// number, times the position wraps where a turn is complete, so the product is the exact remainder of the angle and
// needs no 64-bit floating point, of which this GPU has little; from one of a thread's positions to its next it is an
// addition.  Its upper 32 bits are enough for fp32 results.  The frequencies are the host's, in 64 bits.
// Measured: 131072 x 128 12.9 us (5.2 TB/s); a product and a conversion of 64 bits and sincospif for each pair took 31.7.
#include <math.h>

#include "bd_device.cuh"
#include "bd_internal.h"

namespace bd {
namespace {

constexpr int kThreads = 256;

struct TableArgs {
    float *table;
    unsigned *status;
    int64_t positions;
    int32_t pairs;
    float amplitude;
    uint64_t step[BD_ROTARY_MAX_DIM / 2];  // turns per position, in 2^-64
};

// Of the angle that `phase`, in 2^-32 turns, is: the nearest quarter turn is taken off, the rest is within pi / 4.
__device__ __forceinline__ void cos_sin(uint32_t phase, float amplitude, float &c, float &s) {
    const uint32_t quarter = (phase + (1u << 29)) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(phase - (quarter << 30))) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    const float z = x * x;
    // Taylor's series: the first terms left out are x^11 / 11! < 2^-28 and x^10 / 10! < 2^-25
    float sn = fmaf(z, 1.f / 362880, -1.f / 5040), cs = fmaf(z, 1.f / 40320, -1.f / 720);
    sn = fmaf(z, sn, 1.f / 120), cs = fmaf(z, cs, 1.f / 24);
    sn = fmaf(z, sn, -1.f / 6), cs = fmaf(z, cs, -0.5f);
    sn = fmaf(x * z, sn, x), cs = fmaf(z, cs, 1.f);
    const float u = quarter & 1 ? -sn : cs, v = quarter & 1 ? cs : sn, a = quarter & 2 ? -amplitude : amplitude;
    c = a * u, s = a * v;
}

// kEach pairs of one position per thread, and of positions `rows` apart; a block's threads are whole rows.
template <int kEach>
__global__ void __launch_bounds__(kThreads) rotary_table_kernel(const __grid_constant__ TableArgs a) {
    pdl_trigger_and_wait();
    const int per_row = a.pairs / kEach, rows = kThreads / per_row;
    const int row = threadIdx.x / per_row, at = (threadIdx.x - row * per_row) * kEach;
    if (row >= rows) return;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rows + row, step = static_cast<int64_t>(gridDim.x) * rows;
    uint64_t phase[kEach], add[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) phase[j] = a.step[at + j] * static_cast<uint64_t>(first), add[j] = a.step[at + j] * static_cast<uint64_t>(step);
    float *to = a.table + first * (2 * a.pairs) + at;
    for (int64_t p = first; p < a.positions; p += step, to += step * (2 * a.pairs)) {
        float c[kEach], s[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            cos_sin(static_cast<uint32_t>((phase[j] + (uint64_t{1} << 31)) >> 32), a.amplitude, c[j], s[j]);
            phase[j] += add[j];
        }
        if (!in_bounds(p < a.positions && at + kEach <= a.pairs, a.status)) continue;
        if constexpr (kEach == 4) {
            __stcs(reinterpret_cast<float4 *>(to), make_float4(c[0], c[1], c[2], c[3]));
            __stcs(reinterpret_cast<float4 *>(to + a.pairs), make_float4(s[0], s[1], s[2], s[3]));
        } else {
            to[0] = c[0];
            to[a.pairs] = s[0];
        }
    }
}

}  // namespace

bool rotary_steps(uint64_t *step, int32_t dim, double base, double factor, double original, double low, double high) {
    for (int32_t i = 0; i < dim / 2; ++i) {
        double turns = pow(base, -2.0 * i / dim) / (2 * M_PI);
        double keep = (original * turns - low) / (high - low);
        keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
        turns *= keep + (1 - keep) / factor;
        if (!(turns - turns == 0)) return false;
        step[i] = static_cast<uint64_t>((turns - floor(turns)) * 0x1p64);  // below 2^64: a double below 1 is at most 1 - 2^-53
    }
    return true;
}

cudaError_t launch_rotary_table(float *table, int64_t positions, int32_t dim, const uint64_t *step, float amplitude,
                                const DevCtx &ctx, cudaStream_t stream) {
    TableArgs a;
    a.table = table;
    a.status = ctx.status;
    a.positions = positions;
    a.pairs = dim / 2;
    a.amplitude = amplitude;
    for (int i = 0; i < BD_ROTARY_MAX_DIM / 2; ++i) a.step[i] = i < a.pairs ? step[i] : 0;
    const bool wide = dim % 8 == 0;
    const int rows = kThreads / (a.pairs / (wide ? 4 : 1));
    const int64_t blocks = (positions + rows - 1) / rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 8 * ctx.num_sms ? blocks : 8 * ctx.num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, wide ? rotary_table_kernel<4> : rotary_table_kernel<1>, a);
}

}  // namespace bd
