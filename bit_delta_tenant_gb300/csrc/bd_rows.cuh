// bd_rows.cuh -- 16-byte pieces of bf16 rows as fp32, and back.
#pragma once

#include "bd_device.cuh"

namespace bd {

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    f[0] = bf16lo_to_f32(v.x), f[1] = bf16hi_to_f32(v.x);
    f[2] = bf16lo_to_f32(v.y), f[3] = bf16hi_to_f32(v.y);
    f[4] = bf16lo_to_f32(v.z), f[5] = bf16hi_to_f32(v.z);
    f[6] = bf16lo_to_f32(v.w), f[7] = bf16hi_to_f32(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {  // rounded to nearest
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

}  // namespace bd
