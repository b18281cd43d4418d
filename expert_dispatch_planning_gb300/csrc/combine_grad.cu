// combine_grad.cu -- gradient of the weighted combine (sm_103a).
//
// out[s] = sum_k w[s,k] * y[slot(s,k)] gives dy[slot(s,k)] = w[s,k] * dout[s]
// and dw[s,k] = <dout[s], y[slot(s,k)]>.  Memory bound: dout is read once,
// y read once, dy written once.  A block takes a token: each thread holds a
// 16-byte chunk of dout and goes over the token's K rows with it, keeping a
// partial dot product for each; the block joins them in a fixed order.
// Further blocks zero the groups' padding rows.
#include "vec8.cuh"

namespace moe {

struct CombineGradArgs {
    const uint16_t* dout;
    const uint16_t* y;
    const float* w;
    const int32_t* dst;
    const int32_t* zfr;
    int32_t* status;
    int N, K, H, E;
    int64_t rows;
    uint16_t* dy;
    float* dw;
};

constexpr int kMaxK = 32;

template <int KT>  // K at compile time, or 0 for any K <= 32 (four rows at a time)
__global__ void combine_grad_kernel(const CombineGradArgs a) {
    __shared__ float sums[kMaxK][9];
    pdl_wait();
    pdl_trigger();
    if (ld_volatile_s32(a.status) != 0) return;
    const int64_t H = a.H;
    const int nvec = a.H / 8;
    if (static_cast<int64_t>(blockIdx.x) >= a.N) {  // zero one expert's padding rows
        const int e = static_cast<int>(blockIdx.x - a.N);
        const int64_t first = __ldg(a.zfr + 2 * e), count = __ldg(a.zfr + 2 * e + 1);
        if (count <= 0) return;
        if (first < 0 || first + count > a.rows) {
            if (threadIdx.x == 0) record_error(a.status, MOE_ERR_DEVICE_INDEX, static_cast<int>(first));
            return;
        }
        for (int64_t i = threadIdx.x; i < count * nvec; i += blockDim.x)
            st_v4(a.dy + first * H + 8 * i, make_uint4(0u, 0u, 0u, 0u));
        return;
    }
    const int64_t s = blockIdx.x;
    const int K = KT > 0 ? KT : a.K;
    constexpr int KB = KT > 0 ? KT : 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    bool bad = false;
    for (int k = 0; k < K; ++k) {
        const int64_t raw = raw_slot(__ldg(a.dst + s * K + k));
        bad |= raw < 0 || raw >= a.rows;
    }
    if (bad) {
        if (threadIdx.x == 0) record_error(a.status, MOE_ERR_DEVICE_INDEX, static_cast<int>(s));
        return;
    }
    for (int k0 = 0; k0 < K; k0 += KB) {
        int64_t row[KB];
        float w[KB], dot[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            dot[k] = 0.f;
            row[k] = 0;
            w[k] = 0.f;
            if (k0 + k < K) {
                row[k] = raw_slot(__ldg(a.dst + s * K + k0 + k)) * H;
                w[k] = __ldg(a.w + s * K + k0 + k);
            }
        }
        for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
            float d[8];
            load8(a.dout + s * H, c, d);
            uint4 v[KB];
#pragma unroll
            for (int k = 0; k < KB; ++k)
                if (k0 + k < K) v[k] = ld_stream_v4(a.y + row[k] + 8 * static_cast<int64_t>(c));
#pragma unroll
            for (int k = 0; k < KB; ++k)
                if (k0 + k < K) {
                    float f[8], g[8];
                    unpack8(v[k], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dot[k] = fmaf(d[j], f[j], dot[k]);
                        g[j] = w[k] * d[j];
                    }
                    store8(a.dy + row[k], c, g);
                }
        }
#pragma unroll
        for (int k = 0; k < KB; ++k)
            if (k0 + k < K) {
                const float t = warp_sum(dot[k]);
                if (lane == 0) sums[k0 + k][warp] = t;
            }
    }
    __syncthreads();
    if (threadIdx.x < K) {
        float t = 0.f;
        for (int i = 0; i < warps; ++i) t += sums[threadIdx.x][i];
        a.dw[s * K + threadIdx.x] = t;
    }
}

}  // namespace moe

extern "C" MOE_API int moe_combine_backward(const uint16_t* dout, const uint16_t* y, const float* topk_w, int N, int K,
                                            int H, int E, int64_t rows, const MoePlanOut* plan, uint16_t* dy,
                                            float* dw, cudaStream_t stream) {
    if (plan == nullptr || plan->status == nullptr ||
        (N > 0 && (dout == nullptr || y == nullptr || topk_w == nullptr || dy == nullptr || dw == nullptr ||
                   plan->dst == nullptr || plan->zero_fill_ranges == nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (N < 0 || K < 1 || K > moe::kMaxK || E < 1 || E > 1024 || K > E || H < 8 || H % 8 != 0 || rows < 0 ||
        rows >= (int64_t(1) << 31))
        return MOE_ERR_INVALID_ARG;
    auto aligned = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(topk_w, 4) || !aligned(dw, 4) ||
        !aligned(plan->dst, 4) || !aligned(plan->zero_fill_ranges, 4))
        return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(N) + E >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
    if (N == 0) return MOE_OK;
    const moe::CombineGradArgs a = {dout, y, topk_w, plan->dst, plan->zero_fill_ranges, plan->status,
                                    N,    K, H,      E,         rows,                   dy,           dw};
    int threads = (H / 8 + 31) / 32 * 32;
    if (threads > 256) threads = 256;
    const dim3 grid(static_cast<unsigned>(N + E)), block(static_cast<unsigned>(threads));
    switch (K) {
        case 1: return moe_host::launch(moe::combine_grad_kernel<1>, grid, block, 0, stream, a);
        case 2: return moe_host::launch(moe::combine_grad_kernel<2>, grid, block, 0, stream, a);
        case 4: return moe_host::launch(moe::combine_grad_kernel<4>, grid, block, 0, stream, a);
        case 8: return moe_host::launch(moe::combine_grad_kernel<8>, grid, block, 0, stream, a);
        default: return moe_host::launch(moe::combine_grad_kernel<0>, grid, block, 0, stream, a);
    }
}
