// rotary.cu -- table of rotary positions, scaled for long contexts.
//
//   table[p, i] = amplitude cos(p f_i),  table[p, d + i] = amplitude sin(p f_i)
//
// Bound: HBM (the table is written once).  Angles are whole numbers of 2^-64 turns: a pair's turns per position, as such a
// number, times the position wraps where a turn is complete, so the product is the exact remainder of the angle and
// needs no 64-bit floating point, of which this GPU has little.  The nearest quarter turn is taken off as a whole number
// too, so that what is converted to fp32 is at most an eighth of a turn.  The frequencies are the host's, in 64 bits.
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

__device__ __forceinline__ void cos_sin(uint64_t phase, float amplitude, float &c, float &s) {
    const uint64_t quarter = (phase + (uint64_t{1} << 61)) >> 62;
    const int64_t rest = static_cast<int64_t>(phase - (quarter << 62));  // within an eighth of a turn
    float sn, cs;
    sincospif(static_cast<float>(rest) * 0x1p-63f, &sn, &cs);
    const float x = quarter & 1 ? -sn : cs, y = quarter & 1 ? cs : sn;
    c = amplitude * (quarter & 2 ? -x : x);
    s = amplitude * (quarter & 2 ? -y : y);
}

// kEach pairs of one position per thread.
template <int kEach>
__global__ void __launch_bounds__(kThreads) rotary_table_kernel(const __grid_constant__ TableArgs a) {
    pdl_trigger_and_wait();
    const int per_row = a.pairs / kEach;
    const int64_t n = a.positions * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t p = i / per_row;
        const int at = static_cast<int>(i - p * per_row) * kEach;
        float c[kEach], s[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) cos_sin(a.step[at + j] * static_cast<uint64_t>(p), a.amplitude, c[j], s[j]);
        float *row = a.table + p * (2 * a.pairs) + at;
        if (!in_bounds(p < a.positions && at + kEach <= a.pairs, a.status)) continue;
        if constexpr (kEach == 4) {
            *reinterpret_cast<float4 *>(row) = make_float4(c[0], c[1], c[2], c[3]);
            *reinterpret_cast<float4 *>(row + a.pairs) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            row[0] = c[0];
            row[a.pairs] = s[0];
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
    const int64_t n = positions * (a.pairs / (wide ? 4 : 1)), blocks = (n + kThreads - 1) / kThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 16 * ctx.num_sms ? blocks : 16 * ctx.num_sms));
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
