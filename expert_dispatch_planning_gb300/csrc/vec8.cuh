// vec8.cuh -- eight row elements at a time, held in fp32: bf16 rows as one
// 16-byte vector, fp32 rows as two.
#pragma once

#include <cuda_bf16.h>

#include "moe_common.cuh"

namespace moe {

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Chunk c (elements 8c .. 8c+7) of a row.
__device__ __forceinline__ void load8(const uint16_t* row, int c, float (&f)[8]) {
    unpack8(ld_stream_v4(row + 8 * static_cast<int64_t>(c)), f);
}
__device__ __forceinline__ void load8(const float* row, int c, float (&f)[8]) {
    const float4 a = ld_stream_f4(row + 8 * static_cast<int64_t>(c));
    const float4 b = ld_stream_f4(row + 8 * static_cast<int64_t>(c) + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* row, int c, const float (&f)[8]) {
    st_v4(row + 8 * static_cast<int64_t>(c),
          make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])));
}
__device__ __forceinline__ void store8(float* row, int c, const float (&f)[8]) {
    float4* p = reinterpret_cast<float4*>(row + 8 * static_cast<int64_t>(c));
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}

}  // namespace moe
