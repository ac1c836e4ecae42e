// norm.cu -- residual addition and root-mean-square norm of a batch of rows,
// with per-row choice of the norm weights and bf16 or 8-bit output.
//
//   h = x + r,  y_j = h_j * rsqrt(sum h^2 / n + eps) * w_j
//
// Bound: HBM.  Every input is read once and every output written once (8 bytes
// per element with a residual in bf16), so a row is held in registers between
// the sum and the scaling.  Up to 1024 threads hold a row in 16-byte pieces of 8
// elements, and CTAs take several short rows (one row of 512 to a CTA measured
// 132 us where four take 77: bound by starting CTAs).  The sum of squares goes
// through the warp by shuffles and across warps through shared memory, in an order
// fixed by the row's length.  16 neighbouring lanes hold 128 columns, which is the
// unit of the 8-bit scales.  Measured on 64 Mi elements with residual, bf16: rows of
// 512 79 us and of 4096 80 (the copy rate), 8192 84, 14336 99, 28672 107; 8 bits, rows
// of 4096, 80.
#include <cuda_fp8.h>

#include "bd_device.cuh"
#include "bd_internal.h"
#include "bd_rows.cuh"

namespace bd {
namespace {

constexpr float kTiny = 7.888609e-31f;  // 2^-100

struct NormArgs {
    const uint8_t *x, *residual, *weight;  // bf16 rows
    const int32_t *ids;
    uint8_t *y, *residual_out;
    float *y_scale;
    unsigned *status;
    int64_t m;
    int32_t n, n_weights, row_scale;  // row_scale: one scale per row instead of one per 128 columns
    float eps, inv_n;
};

// A streaming load that is coherent with this kernel's writes: residual_out may be x.
__device__ __forceinline__ uint4 ldg_once(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Sum or maximum over the kWarps warps that share a row, the same value in every thread of theirs.
template <int kWarps, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float *smem) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = kMax ? fmaxf(v, u) : v + u;
    }
    if constexpr (kWarps == 1) return v;
    const int warp = threadIdx.x / 32, first = warp / kWarps * kWarps;
    if (threadIdx.x % 32 == 0) smem[warp] = v;
    __syncthreads();
    float r = smem[first];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) r = kMax ? fmaxf(r, smem[first + w]) : r + smem[first + w];
    return r;
}

// kPerRow threads hold a row, kChunks 16-byte pieces each; kThreads / kPerRow rows to a CTA.
template <int kThreads, int kPerRow, int kChunks, bool kE4m3>
__global__ void __launch_bounds__(kThreads, (kChunks == 1 ? 2048 : kChunks == 2 ? 1536 : 1024) / kThreads) rmsnorm_kernel(const NormArgs a) {
    constexpr int kWarps = kPerRow / 32;
    constexpr bool kLate = kChunks >= 2;  // weights read after the sum: the registers let another CTA onto the SM
    __shared__ float red[2][kThreads / 32];
    pdl_trigger_and_wait();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / kPerRow) + threadIdx.x / kPerRow;
    const int lane = threadIdx.x % kPerRow;
    int32_t id = -1;
    if (row < a.m) {
        id = a.ids ? a.ids[row] : 0;
        if (id >= a.n_weights) id = -1;
        if (id < 0 && lane == 0) flag_status(a.status, kDevBadVariant);
    }
    const int chunks = id >= 0 && in_bounds(row < a.m && id < a.n_weights, a.status) ? a.n / 8 : 0;  // a row beyond the last or with a bad id: nothing is read or written
    const int64_t base = row * a.n * 2;
    [[maybe_unused]] auto in_rows = [&](int c) { return in_bounds(row * a.n + c * 8 + 8 <= a.m * a.n, a.status); };
    float h[kChunks][8];
    uint4 w[kChunks];
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        const int c = lane + u * kPerRow;
        uint4 xv = make_uint4(0, 0, 0, 0), rv = make_uint4(0, 0, 0, 0);
        if (c < chunks) {
            xv = ldg_once(a.x + base + c * 16);
            if (a.residual) rv = *reinterpret_cast<const uint4 *>(a.residual + base + c * 16);
            if (!kLate) w[u] = ldg_keep(a.weight + static_cast<int64_t>(id) * a.n * 2 + c * 16);
        }
        float r[8];
        unpack8(xv, h[u]);
        unpack8(rv, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (a.residual) h[u][j] += r[j];
            ss = fmaf(h[u][j], h[u][j], ss);
        }
        if (c < chunks && a.residual_out && in_rows(c)) *reinterpret_cast<uint4 *>(a.residual_out + base + c * 16) = pack8(h[u]);
    }
    // Divided by n before the reduction, and where a thread's own squares pass fp32 (an element beyond 1.8e19) each of
    // them before it is added, so that only a mean beyond fp32 overflows.  Not always so: squares of less than n 2^-126,
    // which matter where eps is 0, would lose digits.
    float mean = ss * a.inv_n;
    if (!(ss < INFINITY)) {
        mean = 0.f;
#pragma unroll
        for (int u = 0; u < kChunks; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) mean = fmaf(h[u][j] * a.inv_n, h[u][j], mean);
    }
    const float rstd = rsqrtf(row_reduce<kWarps, false>(mean, red[0]) + a.eps);
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        const int c = lane + u * kPerRow;
        float g[8];
        if (kLate && c < chunks) w[u] = ldg_keep(a.weight + static_cast<int64_t>(id) * a.n * 2 + c * 16);
        unpack8(c < chunks ? w[u] : make_uint4(0, 0, 0, 0), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[u][j] = kE4m3 ? h[u][j] * g[j] : h[u][j] * rstd * g[j];
        if constexpr (!kE4m3) {
            if (c < chunks && in_rows(c)) *reinterpret_cast<uint4 *>(a.y + base + c * 16) = pack8(h[u]);
        } else if (a.row_scale) {
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(h[u][j]));
        }
    }
    if constexpr (kE4m3) {
        // The norm's factor is the same for y and for max|y|, so it cancels in y / s: q comes from
        // h w and its maximum alone, in three roundings, and only s sees the factor.
        if (a.row_scale) top = row_reduce<kWarps, true>(top, red[1]);
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int c = lane + u * kPerRow;
            if (!a.row_scale) {
                top = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(h[u][j]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            }
            // scale 1 where everything is (next to) zero, so that no reciprocal overflows
            const bool some = top >= kTiny;
            const float s = some ? __fdiv_rn(top * rstd, 448.f) : 1.f;
            const float inv = some ? __fdiv_rn(448.f, top) : rstd;
            if (c >= chunks || !in_rows(c)) continue;
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q[j] = __nv_cvt_float2_to_fp8x2(make_float2(h[u][2 * j] * inv, h[u][2 * j + 1] * inv), __NV_SATFINITE,
                                                __NV_E4M3);
            *reinterpret_cast<uint2 *>(a.y + row * a.n + c * 8) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
            if (a.row_scale) {
                if (c == 0) a.y_scale[row] = s;
            } else if (c % 16 == 0) {
                a.y_scale[row * (a.n / 128) + c / 16] = s;
            }
        }
    }
}

template <int kThreads, int kPerRow, int kChunks>
cudaError_t launch_sized(const NormArgs &a, bool e4m3, cudaStream_t stream) {
    constexpr int kRows = kThreads / kPerRow;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.m + kRows - 1) / kRows));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return e4m3 ? cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kThreads, kPerRow, kChunks, true>, a)
                : cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kThreads, kPerRow, kChunks, false>, a);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormProblem &p, const DevCtx &ctx, cudaStream_t stream) {
    NormArgs a;
    a.x = static_cast<const uint8_t *>(p.x);
    a.residual = static_cast<const uint8_t *>(p.residual);
    a.weight = static_cast<const uint8_t *>(p.weight);
    a.ids = p.ids;
    a.y = static_cast<uint8_t *>(p.y);
    a.residual_out = static_cast<uint8_t *>(p.residual_out);
    a.y_scale = p.y_scale;
    a.status = ctx.status;
    a.m = p.m;
    a.n = static_cast<int32_t>(p.n);
    a.n_weights = p.n_weights;
    a.row_scale = p.scale_cols != 128;
    a.eps = p.eps;
    a.inv_n = 1.f / static_cast<float>(p.n);
    const bool e4m3 = p.y_type == BD_Y_E4M3;
    if (p.n <= 256) return launch_sized<256, 32, 1>(a, e4m3, stream);
    if (p.n <= 512) return launch_sized<256, 64, 1>(a, e4m3, stream);
    if (p.n <= 1024) return launch_sized<256, 128, 1>(a, e4m3, stream);
    if (p.n <= 2048) return launch_sized<256, 256, 1>(a, e4m3, stream);
    if (p.n <= 4096) return launch_sized<512, 512, 1>(a, e4m3, stream);
    if (p.n <= 8192) return launch_sized<512, 512, 2>(a, e4m3, stream);
    if (p.n <= 16384) return launch_sized<512, 512, 4>(a, e4m3, stream);
    return launch_sized<1024, 1024, 4>(a, e4m3, stream);
}

}  // namespace bd
