// attention_scored.cu -- attention.cuh's kernels for scores with a rule, caches of bf16 and 8 bits.
#include "attention.cuh"

namespace bd {
namespace {

template <int kDim>
cudaError_t launch_dim(const AttnArgs &a, int type, bool pack, const DevCtx &ctx, cudaStream_t stream) {
    if (type == kE4m3Type)
        return pack ? launch_typed<kDim, kE4m3Type, true, true>(a, ctx, stream) : launch_typed<kDim, kE4m3Type, false, true>(a, ctx, stream);
    return pack ? launch_typed<kDim, kBf16, true, true>(a, ctx, stream) : launch_typed<kDim, kBf16, false, true>(a, ctx, stream);
}

}  // namespace

cudaError_t launch_attention_scored(const AttnArgs &a, int type, int dim, bool pack, const DevCtx &ctx, cudaStream_t stream) {
    return dim == 128 ? launch_dim<128>(a, type, pack, ctx, stream) : launch_dim<64>(a, type, pack, ctx, stream);
}

}  // namespace bd
