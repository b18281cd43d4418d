// norm_parts.cuh -- what the kernels of norm.cu and block_norm.cu share: sums
// and maxima over a row's threads, loads and stores of elements held in fp32,
// the 8-bit output's rounding, and the host's choice of a launch.
#pragma once

#include <cuda_fp8.h>

#include <cmath>

#include "vec8.cuh"

namespace moe {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastEps = 0x1p-100f;  // from here on eps covers what squares lose below the normal numbers

// Sums (or maxima) over the threads that share a row: a warp, or the block
// through shared memory.  `buf` holds 32 floats; the leading barrier lets it
// be used again.
template <bool WARP, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float t = __shfl_xor_sync(FULL_MASK, v, o);
        v = MAX ? fmaxf(v, t) : v + t;
    }
    if constexpr (!WARP) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        const int warps = blockDim.x >> 5;
        v = (threadIdx.x & 31) < warps ? buf[threadIdx.x & 31] : 0.f;  // maxima are of magnitudes: 0 is neutral
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float t = __shfl_xor_sync(FULL_MASK, v, o);
            v = MAX ? fmaxf(v, t) : v + t;
        }
    }
    return v;
}

__device__ __forceinline__ void load_weight8(const void* w, int f32, int c, float (&f)[8]) {
    if (f32) {
        const float4* p = reinterpret_cast<const float4*>(w) + 2 * static_cast<int64_t>(c);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8(__ldg(reinterpret_cast<const uint4*>(w) + c), f);
    }
}

// The residual's elements 8c .. 8c+7: residual_out may be the residual itself,
// so that they are not read-only for the kernel.
__device__ __forceinline__ void load8_written(const uint16_t* row, int c, float (&f)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(row + 8 * static_cast<int64_t>(c)), f);
}
__device__ __forceinline__ void load8_written(const float* row, int c, float (&f)[8]) {
    const float4* p = reinterpret_cast<const float4*>(row + 8 * static_cast<int64_t>(c));
    const float4 a = p[0], b = p[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The 8-bit output's scale of a row and its values' rounding: a product with
// the scale's reciprocal, both moved up by a power of two where the reciprocal
// would overflow.
struct Quantum {
    float scale, up, inv;
    __device__ __forceinline__ uint32_t round4(const float* v) const {
        const float2 a = make_float2(v[0] * up * inv, v[1] * up * inv), b = make_float2(v[2] * up * inv, v[3] * up * inv);
        return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
               static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
    }
};
__device__ __forceinline__ Quantum quantum_of(float amax) {
    Quantum q;
    q.scale = fmaxf((amax > 0.f ? amax : 1.f) * (1.f / kE4m3Max), 0x1p-149f);  // never 0
    q.up = q.scale < 1e-30f ? 0x1p64f : 1.f;
    q.inv = __fdividef(1.f, q.scale * q.up);
    return q;
}

// ---------------------------------------------------------------- four elements, the block's sums
__device__ __forceinline__ void load4(const uint16_t* p, float (&f)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// The block's sum or maximum with one barrier: `buf` holds two sets of 32
// floats that a caller uses in turn.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float t = __shfl_xor_sync(FULL_MASK, v, o);
        v = MAX ? fmaxf(v, t) : v + t;
    }
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < (blockDim.x >> 5) ? buf[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float t = __shfl_xor_sync(FULL_MASK, v, o);
        v = MAX ? fmaxf(v, t) : v + t;
    }
    return v;
}

constexpr int kRingThreads = 1024;

}  // namespace moe

// ---------------------------------------------------------------- host
namespace moe_host {

constexpr int kMaxH = 32768;  // a row in the registers of 1024 threads

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool float_type(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }

// chunks of 8 elements a thread, with at most 256 threads a chunk
inline int norm_vpt(int H) { return H <= 2048 ? 1 : H <= 8192 ? 2 : 4; }
inline int norm_threads(int H) { return (H / 8 + 32 * norm_vpt(H) - 1) / (32 * norm_vpt(H)) * 32; }

// Squares are summed scaled down by a power of two near 1/sqrt(H), so that a
// row overflows only where a mean square does; `mean` is 1/(H down^2).
inline void square_scale(int H, float* down, float* mean) {
    int k = 0;
    while ((int64_t(1) << (2 * k)) < H) ++k;
    *down = std::ldexp(1.f, -k);
    *mean = static_cast<float>(static_cast<double>(int64_t(1) << (2 * k)) / H);
}

}  // namespace moe_host
