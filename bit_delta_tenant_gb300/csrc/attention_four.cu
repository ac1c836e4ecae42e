// attention_four.cu -- attention.cuh's kernels for caches of 4 bits.
#include "attention.cuh"

namespace bd {
namespace {

template <int kDim, bool kPack>
cudaError_t launch_scored(const AttnArgs &a, bool scored, const DevCtx &ctx, cudaStream_t stream) {
    return scored ? launch_typed<kDim, kE2m1, kPack, true>(a, ctx, stream) : launch_typed<kDim, kE2m1, kPack, false>(a, ctx, stream);
}

}  // namespace

cudaError_t launch_attention_four(const AttnArgs &a, bool scored, int dim, bool pack, const DevCtx &ctx, cudaStream_t stream) {
    if (dim == 128) return pack ? launch_scored<128, true>(a, scored, ctx, stream) : launch_scored<128, false>(a, scored, ctx, stream);
    return pack ? launch_scored<64, true>(a, scored, ctx, stream) : launch_scored<64, false>(a, scored, ctx, stream);
}

}  // namespace bd
