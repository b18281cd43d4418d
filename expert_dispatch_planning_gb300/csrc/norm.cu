// norm.cu -- root-mean-square norm with the residual's addition and its
// gradient (sm_103a).
//
// Forward, one pass over the row: s = x + r stays in registers (fp32), the
// row's sum of squares gives rstd, v = s * rstd * w is stored as bf16, and
// its largest magnitude gives the scale of the 8-bit output.  Backward: the
// row's mean of dy*w*xhat gives dx; dy*xhat is summed over the rows of a
// block in registers (a thread keeps its columns for all of them), one
// partial row a block, and a second launch adds the partials in block order,
// so that the result does not depend on scheduling.
//
// Memory bound: every element is read once and written once.  Three forms:
//   - H <= 512: a warp a row, four rows a block;
//   - few rows, or very wide ones: a block a row, 8, 16 or 32 elements a thread;
//     (past 8192 columns the gradient spills registers: right, but not tuned);
//   - else a ring: blocks that stay, each thread copying its own columns of the
//     next rows into its own places in shared memory (cp.async) while the block
//     works on a row, so that the row's reductions never empty the memory
//     pipeline.  A thread reads only what it copied, so the ring needs no
//     barrier; the row's sums take one each.
// Measured (GB300, copy rate 6.68 TB/s): forward with a bf16 residual and the
// 8-bit output at 8192 x 7168, 84 us, 6.3 TB/s (a block a row: 95 us; issue
// slots bound it, 66% taken, until the values' divisions became products);
// backward with fp32 sums at 16384 x 4096, 165 us, 6.5 TB/s (a block a row: 228).
#include <cuda_fp8.h>

#include <cmath>

#include "vec8.cuh"

namespace moe {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastEps = 0x1p-100f;  // from here on eps covers what squares lose below the normal numbers

struct NormArgs {
    const uint16_t* x;
    const void* residual;
    const void* weight;
    int weight_f32;
    int N, H;
    float eps;
    float down, mean;  // a power of two near 1/sqrt(H), and 1/(H down^2): the squares are summed scaled down, so
                       // that a row overflows only where a mean square does
    uint16_t* y;
    void* residual_out;
    float* rstd;
    uint8_t* q;
    float* q_scale;
};

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

// RES: 0 no residual, 1 bf16, 2 fp32.
template <int VPT, bool WARP, int RES>
__global__ void __launch_bounds__(WARP ? 128 : 256 * VPT) norm_kernel(const NormArgs a) {
    __shared__ float buf[32];
    pdl_wait();
    pdl_trigger();
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int lanes = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.N) return;
    const int nvec = a.H / 8;
    const int64_t at = row * a.H;

    float s[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * lanes;
        if (c < nvec) {
            load8(a.x + at, c, s[i]);
            if constexpr (RES != 0) {
                float r[8];
                if constexpr (RES == 2) load8_written(static_cast<const float*>(a.residual) + at, c, r);
                else load8_written(static_cast<const uint16_t*>(a.residual) + at, c, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i][j] += r[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = s[i][j] * a.down;
                ss = fmaf(t, t, ss);
            }
        }
    }
    ss = row_reduce<WARP, false>(ss, buf);
    float rstd = rsqrtf(fmaf(ss, a.mean, a.eps));  // within 2^-22
    if (!(fmaf(ss, a.mean, a.eps) >= kLeastEps)) {
        // Squares may have lost digits below the normal numbers, or vanished, and
        // eps does not cover them.  No value is above 2^-42: all are summed again,
        // scaled.  (The row's threads hold the same sum and take the same way.)
        constexpr float kUp = 0x1p90f;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (lane + i * lanes < nvec)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = s[i][j] * kUp;
                    ss = fmaf(t, t, ss);
                }
        ss = row_reduce<WARP, false>(ss, buf) * (a.down * a.down);
        rstd = kUp * rsqrtf(fmaf(ss, a.mean, a.eps * kUp * kUp));
    }
    if (a.rstd != nullptr && lane == 0) a.rstd[row] = rstd;

    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * lanes;
        if (c < nvec) {
            if constexpr (RES == 2) {
                if (a.residual_out != nullptr) store8(static_cast<float*>(a.residual_out) + at, c, s[i]);
            } else if constexpr (RES == 1) {
                if (a.residual_out != nullptr) store8(static_cast<uint16_t*>(a.residual_out) + at, c, s[i]);
            }
            float w[8];
            load_weight8(a.weight, a.weight_f32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[i][j] = s[i][j] * rstd * w[j];
                amax = fmaxf(amax, fabsf(s[i][j]));
            }
            if (a.y != nullptr) store8(a.y + at, c, s[i]);
        }
    }
    if (a.q == nullptr) return;
    amax = row_reduce<WARP, true>(amax, buf);
    const Quantum q = quantum_of(amax);
    if (lane == 0) a.q_scale[row] = q.scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * lanes;
        if (c < nvec)
            *reinterpret_cast<uint2*>(a.q + at + 8 * static_cast<int64_t>(c)) =
                make_uint2(q.round4(s[i]), q.round4(s[i] + 4));
    }
}

// ---------------------------------------------------------------- backward
struct NormBackwardArgs {
    const uint16_t* dy;
    const void* s;
    const void* weight;
    int weight_f32;
    const float* rstd;
    const void* ds;
    int N, H;
    uint16_t* dx;
    float* dres;
    float* partial;  // [gridDim.x][H], or null without dweight
};

template <int VPT, bool WARP, typename S>
__global__ void __launch_bounds__(WARP ? 128 : 256 * VPT) norm_backward_kernel(const NormBackwardArgs a) {
    extern __shared__ float sh[];  // WARP: [warps][H] for the block's sum
    __shared__ float buf[32];
    pdl_wait();
    pdl_trigger();
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int lanes = WARP ? 32 : blockDim.x;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    const int per_step = WARP ? warps : 1;
    const int nvec = a.H / 8;

    float w[VPT][8], acc[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * lanes;
        if (c < nvec) load_weight8(a.weight, a.weight_f32, c, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    }
    // rows of a block are consecutive: its partial sum has a fixed order
    const int64_t steps = (static_cast<int64_t>(a.N) + per_step - 1) / per_step;
    const int64_t begin = blockIdx.x * steps / gridDim.x, end = (blockIdx.x + 1) * steps / gridDim.x;
    for (int64_t step = begin; step < end; ++step) {
        const int64_t row = WARP ? step * per_step + warp : step;
        if (row >= a.N) break;
        const int64_t at = row * a.H;
        const float rstd = __ldg(a.rstd + row);
        float xhat[VPT][8], t[VPT][8], d[VPT][8];  // ds is asked for with the rest, before the row's sum is waited for
        float dot = 0.f;
        if (a.ds != nullptr) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (lane + i * lanes < nvec) load8(static_cast<const S*>(a.ds) + at, lane + i * lanes, d[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) {
                load8(a.dy + at, c, t[i]);
                load8(static_cast<const S*>(a.s) + at, c, xhat[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xhat[i][j] *= rstd;
                    acc[i][j] = fmaf(t[i][j], xhat[i][j], acc[i][j]);
                    t[i][j] *= w[i][j];
                    dot = fmaf(t[i][j], xhat[i][j], dot);
                }
            }
        }
        const float mean = row_reduce<WARP, false>(dot, buf) / static_cast<float>(a.H);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] += rstd * (t[i][j] - xhat[i][j] * mean);
                store8(a.dx + at, c, d[i]);
                if (a.dres != nullptr) store8(a.dres + at, c, d[i]);
            }
        }
    }
    if (a.partial == nullptr) return;
    float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.H;
    if constexpr (WARP) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) store8(sh + warp * a.H, c, acc[i]);
        }
        __syncthreads();
        for (int h = threadIdx.x; h < a.H; h += blockDim.x) {
            float v = 0.f;
            for (int k = 0; k < warps; ++k) v += sh[k * a.H + h];
            out[h] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) store8(out, c, acc[i]);
        }
    }
}

// ---------------------------------------------------------------- ring
// A thread owns groups of four columns, t, t + T, ...: 8 bytes of a bf16 row,
// 16 of an fp32 one, neighbouring threads side by side.
__device__ __forceinline__ void cp_async_group(uint16_t* dst, const uint16_t* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_group(float* dst, const float* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
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
__device__ __forceinline__ void load_weight4(const void* w, int f32, int h, float (&f)[4]) {
    if (f32) load4(static_cast<const float*>(w) + h, f);
    else load4(static_cast<const uint16_t*>(w) + h, f);
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
constexpr int kRingGroups = 2;  // groups of four columns a thread at most: H <= 8192

// R: the residual's element type (uint16_t also stands for none).
template <int SLOTS, typename R, bool RES>
__global__ void __launch_bounds__(kRingThreads) norm_ring_kernel(const NormArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];  // [SLOTS][x row, residual row]
    __shared__ float buf[2][2][32];
    pdl_wait();
    pdl_trigger();
    const int T = blockDim.x, H = a.H;
    const uint32_t slot_bytes = static_cast<uint32_t>(H) * (RES ? 2 + sizeof(R) : 2);
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.N / gridDim.x;
    const int64_t end = (static_cast<int64_t>(blockIdx.x) + 1) * a.N / gridDim.x;
    auto fetch = [&](int64_t row, uint32_t slot) {
        if (row < end) {
            uint16_t* x = reinterpret_cast<uint16_t*>(smem + slot * slot_bytes);
            R* r = reinterpret_cast<R*>(x + H);
#pragma unroll
            for (int i = 0; i < kRingGroups; ++i) {
                const int h = 4 * (threadIdx.x + i * T);
                if (h < H) {
                    cp_async_group(x + h, a.x + row * H + h);
                    if constexpr (RES) cp_async_group(r + h, static_cast<const R*>(a.residual) + row * H + h);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float w[kRingGroups][4];
#pragma unroll
    for (int i = 0; i < kRingGroups; ++i) {
        const int h = 4 * (threadIdx.x + i * T);
        if (h < H) load_weight4(a.weight, a.weight_f32, h, w[i]);
    }
#pragma unroll
    for (int j = 0; j < SLOTS - 1; ++j) fetch(begin + j, j);
    uint32_t slot = 0;  // the row's
    for (int64_t row = begin; row < end; ++row, slot = (slot + 1) % SLOTS) {
        fetch(row + SLOTS - 1, (slot + SLOTS - 1) % SLOTS);
        asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
        const uint16_t* x = reinterpret_cast<const uint16_t*>(smem + slot * slot_bytes);
        const R* r = reinterpret_cast<const R*>(x + H);
        const int64_t at = row * H;
        float(*sums)[32] = buf[row & 1];
        float s[kRingGroups][4];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kRingGroups; ++i) {
            const int h = 4 * (threadIdx.x + i * T);
            if (h < H) {
                load4(x + h, s[i]);
                if constexpr (RES) {
                    float q[4];
                    load4(r + h, q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] += q[j];
                    if (a.residual_out != nullptr) store4(static_cast<R*>(a.residual_out) + at + h, s[i]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float t = s[i][j] * a.down;
                    ss = fmaf(t, t, ss);
                }
            }
        }
        ss = block_reduce<false>(ss, sums[0]);
        const float rstd = rsqrtf(fmaf(ss, a.mean, a.eps));  // within 2^-22
        if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < kRingGroups; ++i) {
            const int h = 4 * (threadIdx.x + i * T);
            if (h < H) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = s[i][j] * rstd * w[i][j];
                    amax = fmaxf(amax, fabsf(s[i][j]));
                }
                if (a.y != nullptr) store4(a.y + at + h, s[i]);
            }
        }
        if (a.q == nullptr) continue;
        amax = block_reduce<true>(amax, sums[1]);
        const Quantum q = quantum_of(amax);
        if (threadIdx.x == 0) a.q_scale[row] = q.scale;
#pragma unroll
        for (int i = 0; i < kRingGroups; ++i) {
            const int h = 4 * (threadIdx.x + i * T);
            if (h < H)
                *reinterpret_cast<uint32_t*>(a.q + at + h) = q.round4(s[i]);
        }
    }
}

template <int SLOTS, typename S, bool DS>
__global__ void __launch_bounds__(kRingThreads) norm_backward_ring_kernel(const NormBackwardArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];  // [SLOTS][dy row, s row, ds row]
    __shared__ float buf[2][32];
    pdl_wait();
    pdl_trigger();
    const int T = blockDim.x, H = a.H;
    const uint32_t slot_bytes = static_cast<uint32_t>(H) * (2 + (DS ? 2 : 1) * sizeof(S));
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.N / gridDim.x;
    const int64_t end = (static_cast<int64_t>(blockIdx.x) + 1) * a.N / gridDim.x;
    auto fetch = [&](int64_t row, uint32_t slot) {
        if (row < end) {
            uint16_t* dy = reinterpret_cast<uint16_t*>(smem + slot * slot_bytes);
            S* s = reinterpret_cast<S*>(dy + H);
#pragma unroll
            for (int i = 0; i < kRingGroups; ++i) {
                const int h = 4 * (threadIdx.x + i * T);
                if (h < H) {
                    cp_async_group(dy + h, a.dy + row * H + h);
                    cp_async_group(s + h, static_cast<const S*>(a.s) + row * H + h);
                    if constexpr (DS) cp_async_group(s + H + h, static_cast<const S*>(a.ds) + row * H + h);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float w[kRingGroups][4], acc[kRingGroups][4];
#pragma unroll
    for (int i = 0; i < kRingGroups; ++i) {
        const int h = 4 * (threadIdx.x + i * T);
        if (h < H) load_weight4(a.weight, a.weight_f32, h, w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < SLOTS - 1; ++j) fetch(begin + j, j);
    uint32_t slot = 0;  // the row's
    float next_rstd = begin < end ? __ldg(a.rstd + begin) : 0.f;
    for (int64_t row = begin; row < end; ++row, slot = (slot + 1) % SLOTS) {
        fetch(row + SLOTS - 1, (slot + SLOTS - 1) % SLOTS);
        const float rstd = next_rstd;
        if (row + 1 < end) next_rstd = __ldg(a.rstd + row + 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
        const uint16_t* dy = reinterpret_cast<const uint16_t*>(smem + slot * slot_bytes);
        const S* s = reinterpret_cast<const S*>(dy + H);
        const int64_t at = row * H;
        float xhat[kRingGroups][4], t[kRingGroups][4];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kRingGroups; ++i) {
            const int h = 4 * (threadIdx.x + i * T);
            if (h < H) {
                load4(dy + h, t[i]);
                load4(s + h, xhat[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    xhat[i][j] *= rstd;
                    acc[i][j] = fmaf(t[i][j], xhat[i][j], acc[i][j]);
                    t[i][j] *= w[i][j];
                    dot = fmaf(t[i][j], xhat[i][j], dot);
                }
            }
        }
        const float mean = block_reduce<false>(dot, buf[row & 1]) / static_cast<float>(H);
#pragma unroll
        for (int i = 0; i < kRingGroups; ++i) {
            const int h = 4 * (threadIdx.x + i * T);
            if (h < H) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                if constexpr (DS) load4(s + H + h, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] += rstd * (t[i][j] - xhat[i][j] * mean);
                store4(a.dx + at + h, d);
                if (a.dres != nullptr) store4(a.dres + at + h, d);
            }
        }
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int i = 0; i < kRingGroups; ++i) {
        const int h = 4 * (threadIdx.x + i * T);
        if (h < H) store4(a.partial + static_cast<int64_t>(blockIdx.x) * H + h, acc[i]);
    }
}

// dweight[h] = sum of the blocks' partials: 32 columns a block; each of its 32
// warps adds every 32nd partial, and the warps' sums are joined in order.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* partial, int blocks, int H, float* dweight) {
    __shared__ float sh[32][33];
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x * 32 + threadIdx.x, g = threadIdx.y;
    float v = 0.f;
    if (h < H) {
#pragma unroll 4
        for (int b = g; b < blocks; b += 32) v += partial[static_cast<int64_t>(b) * H + h];
    }
    sh[g][threadIdx.x] = v;
    __syncthreads();
    v = warp_sum(sh[threadIdx.x][g]);  // warp g joins column g
    if (threadIdx.x == 0 && blockIdx.x * 32 + g < H) dweight[blockIdx.x * 32 + g] = v;
}

}  // namespace moe

// ---------------------------------------------------------------- host
namespace {

constexpr int kMaxH = 32768;  // a row in the registers of 1024 threads

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool float_type(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }

// chunks of 8 elements a thread, with at most 256 threads a chunk
int norm_vpt(int H) { return H <= 2048 ? 1 : H <= 8192 ? 2 : 4; }
int norm_threads(int H) { return (H / 8 + 32 * norm_vpt(H) - 1) / (32 * norm_vpt(H)) * 32; }

template <int VPT, bool WARP>
int launch_norm(const moe::NormArgs& a, int res, dim3 grid, dim3 block, cudaStream_t stream) {
    if (res == 0) return moe_host::launch(moe::norm_kernel<VPT, WARP, 0>, grid, block, 0, stream, a);
    if (res == 1) return moe_host::launch(moe::norm_kernel<VPT, WARP, 1>, grid, block, 0, stream, a);
    return moe_host::launch(moe::norm_kernel<VPT, WARP, 2>, grid, block, 0, stream, a);
}

template <int VPT, bool WARP>
int launch_backward(const moe::NormBackwardArgs& a, bool f32, dim3 grid, dim3 block, size_t smem,
                    cudaStream_t stream) {
    if (f32) return moe_host::launch(moe::norm_backward_kernel<VPT, WARP, float>, grid, block, smem, stream, a);
    return moe_host::launch(moe::norm_backward_kernel<VPT, WARP, uint16_t>, grid, block, smem, stream, a);
}

// The ring form: `slot` bytes a row, two to eight slots, blocks as many as
// their rings and threads fit an SM.  Taken when every block gets a few rows
// (fewer would only wait for their own) and a row has enough columns to keep
// its barrier cheap.  The forward kernel's is not taken with an eps (0, say) that does
// not cover vanishing squares: the ring has no second sum, since a branch in
// its loop costs up to a fifth (16384 x 1024: 16.6 us without, 19.6 us with it).
struct Ring {
    int slots = 0, threads = 0, blocks = 0;  // slots = 0: not taken
    size_t smem = 0;
};
Ring ring_for(int N, int H, size_t slot) {
    constexpr size_t kSmem = 220 * 1024;
    Ring r;
    if (H <= 512 || H > 4 * moe::kRingGroups * moe::kRingThreads || 2 * slot > kSmem) return r;
    const int slots = 8 * slot <= kSmem / 2 ? 8 : 4 * slot <= kSmem ? 4 : 2;
    const int per_thread = 4 * moe::kRingGroups;
    const int threads = (H + 32 * per_thread - 1) / (32 * per_thread) * 32;
    const int by_smem = static_cast<int>(kSmem / (slots * slot)), by_threads = 1536 / threads;
    const int per_sm = by_smem < by_threads ? by_smem : by_threads;
    const int blocks = moe_host::num_sms() * (per_sm < 1 ? 1 : per_sm > 6 ? 6 : per_sm);
    if (N < 4 * blocks) return r;
    r.slots = slots;
    r.threads = threads;
    r.blocks = blocks;
    r.smem = slots * slot;
    return r;
}

template <typename Kernel, typename Args>
int launch_ring(Kernel kernel, const Ring& r, const Args& a, cudaStream_t stream) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) != cudaSuccess)
        return MOE_ERR_CUDA;
    return moe_host::launch(kernel, dim3(static_cast<unsigned>(r.blocks)), dim3(static_cast<unsigned>(r.threads)), r.smem,
                            stream, a);
}

template <int SLOTS>
int launch_norm_ring(const Ring& r, const moe::NormArgs& a, int res, cudaStream_t stream) {
    if (res == 0) return launch_ring(moe::norm_ring_kernel<SLOTS, uint16_t, false>, r, a, stream);
    if (res == 1) return launch_ring(moe::norm_ring_kernel<SLOTS, uint16_t, true>, r, a, stream);
    return launch_ring(moe::norm_ring_kernel<SLOTS, float, true>, r, a, stream);
}

template <int SLOTS>
int launch_backward_ring(const Ring& r, const moe::NormBackwardArgs& a, bool f32, cudaStream_t stream) {
    if (f32)
        return a.ds != nullptr ? launch_ring(moe::norm_backward_ring_kernel<SLOTS, float, true>, r, a, stream)
                               : launch_ring(moe::norm_backward_ring_kernel<SLOTS, float, false>, r, a, stream);
    return a.ds != nullptr ? launch_ring(moe::norm_backward_ring_kernel<SLOTS, uint16_t, true>, r, a, stream)
                           : launch_ring(moe::norm_backward_ring_kernel<SLOTS, uint16_t, false>, r, a, stream);
}

// Blocks of the backward kernel's other forms: four an SM, no more than there are rows.
int backward_blocks(int N, int H) {
    const int64_t units = H <= 512 ? (static_cast<int64_t>(N) + 3) / 4 : N;
    const int64_t cap = static_cast<int64_t>(moe_host::num_sms()) * 4;
    return static_cast<int>(units < cap ? units : cap);
}

}  // namespace

extern "C" MOE_API int moe_residual_norm(const uint16_t* x, const void* residual, int residual_dtype,
                                         const void* weight, int weight_dtype, int N, int H, float eps, uint16_t* y,
                                         void* residual_out, float* rstd, uint8_t* q, float* q_scale,
                                         cudaStream_t stream) {
    if (N < 0 || H < 8 || H % 8 != 0 || !(eps >= 0.f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (!float_type(weight_dtype) || (residual != nullptr && !float_type(residual_dtype))) return MOE_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_scale == nullptr) && N > 0) return MOE_ERR_INVALID_ARG;
    if (N > 0 && (x == nullptr || weight == nullptr || (y == nullptr && q == nullptr))) return MOE_ERR_INVALID_ARG;
    if (residual == nullptr && residual_out != nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(y) || !aligned16(residual_out) ||
        (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0 || (reinterpret_cast<uintptr_t>(q) & 7u) != 0 ||
        (reinterpret_cast<uintptr_t>(q_scale) & 3u) != 0)
        return MOE_ERR_INVALID_ARG;
    if (H > kMaxH) return MOE_ERR_UNSUPPORTED;
    if (N == 0) return MOE_OK;
    int k = 0;
    while ((int64_t(1) << (2 * k)) < H) ++k;
    const float mean = static_cast<float>(static_cast<double>(int64_t(1) << (2 * k)) / H);
    const moe::NormArgs a = {x, residual, weight,       weight_dtype == MOE_DTYPE_F32, N, H, eps, std::ldexp(1.f, -k),
                             mean, y,     residual_out, rstd,                          q, q_scale};
    const int res = residual == nullptr ? 0 : residual_dtype == MOE_DTYPE_F32 ? 2 : 1;
    const Ring ring = eps >= moe::kLeastEps ? ring_for(N, H, static_cast<size_t>(H) * (2 + 2 * res)) : Ring();
    // (four slots of at most 8192 columns in 6 bytes always fit)
    if (ring.slots == 8) return launch_norm_ring<8>(ring, a, res, stream);
    if (ring.slots == 4) return launch_norm_ring<4>(ring, a, res, stream);
    if (H <= 512) {
        const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(N) + 3) / 4)), block(128);
        return H <= 256 ? launch_norm<1, true>(a, res, grid, block, stream)
                        : launch_norm<2, true>(a, res, grid, block, stream);
    }
    const dim3 grid(static_cast<unsigned>(N)), block(static_cast<unsigned>(norm_threads(H)));
    switch (norm_vpt(H)) {
        case 1: return launch_norm<1, false>(a, res, grid, block, stream);
        case 2: return launch_norm<2, false>(a, res, grid, block, stream);
        default: return launch_norm<4, false>(a, res, grid, block, stream);
    }
}

extern "C" MOE_API size_t moe_residual_norm_backward_workspace_size(int N, int H) {
    if (N < 0 || H < 8 || H % 8 != 0 || H > kMaxH) return 0;
    int blocks = backward_blocks(N, H);  // the ring form may have more, of the narrowest type
    if (N > blocks) blocks = N < 6 * moe_host::num_sms() ? N : 6 * moe_host::num_sms();
    return static_cast<size_t>(blocks > 0 ? blocks : 1) * H * sizeof(float);
}

extern "C" MOE_API int moe_residual_norm_backward(const uint16_t* dy, const void* s, int s_dtype, const void* weight,
                                                  int weight_dtype, const float* rstd, const void* ds, int N, int H,
                                                  uint16_t* dx, float* dres, float* dweight, void* workspace,
                                                  size_t workspace_bytes, cudaStream_t stream) {
    if (N < 0 || H < 8 || H % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (!float_type(weight_dtype) || !float_type(s_dtype)) return MOE_ERR_INVALID_ARG;
    if (N > 0 && (dy == nullptr || s == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr))
        return MOE_ERR_INVALID_ARG;
    if (dres != nullptr && s_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(s) || !aligned16(weight) || !aligned16(ds) || !aligned16(dx) ||
        !aligned16(dres) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(dweight) & 3u) != 0)
        return MOE_ERR_INVALID_ARG;
    if (H > kMaxH) return MOE_ERR_UNSUPPORTED;
    if (dweight != nullptr && N > 0) {
        if (workspace == nullptr) return MOE_ERR_INVALID_ARG;
        if (workspace_bytes < moe_residual_norm_backward_workspace_size(N, H)) return MOE_ERR_CAPACITY;
    }
    if (N == 0) {
        if (dweight != nullptr && cudaMemsetAsync(dweight, 0, sizeof(float) * H, stream) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    const bool f32 = s_dtype == MOE_DTYPE_F32;
    const size_t esize = f32 ? 4 : 2;
    const Ring ring = ring_for(N, H, H * (2 + (ds != nullptr ? 2 : 1) * esize));
    const int blocks = ring.slots > 0 ? ring.blocks : backward_blocks(N, H);
    const moe::NormBackwardArgs a = {dy, s, weight, weight_dtype == MOE_DTYPE_F32, rstd, ds, N, H, dx, dres,
                                     dweight != nullptr ? static_cast<float*>(workspace) : nullptr};
    const dim3 grid(static_cast<unsigned>(blocks));
    int rc;
    if (ring.slots > 0) {
        rc = ring.slots == 8   ? launch_backward_ring<8>(ring, a, f32, stream)
             : ring.slots == 4 ? launch_backward_ring<4>(ring, a, f32, stream)
                               : launch_backward_ring<2>(ring, a, f32, stream);
    } else if (H <= 512) {
        const dim3 block(128);
        const size_t smem = 4 * sizeof(float) * H;
        rc = H <= 256 ? launch_backward<1, true>(a, f32, grid, block, smem, stream)
                      : launch_backward<2, true>(a, f32, grid, block, smem, stream);
    } else {
        const dim3 block(static_cast<unsigned>(norm_threads(H)));
        switch (norm_vpt(H)) {
            case 1: rc = launch_backward<1, false>(a, f32, grid, block, 0, stream); break;
            case 2: rc = launch_backward<2, false>(a, f32, grid, block, 0, stream); break;
            default: rc = launch_backward<4, false>(a, f32, grid, block, 0, stream); break;
        }
    }
    if (rc != MOE_OK || dweight == nullptr) return rc;
    return moe_host::launch(moe::norm_dweight_kernel, dim3(static_cast<unsigned>((H + 31) / 32)), dim3(32, 32), 0,
                            stream, static_cast<const float*>(a.partial), blocks, H, dweight);
}
