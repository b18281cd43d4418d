// combine_grad.cu -- gradient of the weighted combine (sm_103a).
//
// out[s] = sum_k w[s,k] * y[slot(s,k)] gives dy[slot(s,k)] = w[s,k] * dout[s]
// and dw[s,k] = <dout[s], y[slot(s,k)]>.  Memory bound: dout is read once,
// y read once, dy written once.  1, 2, 4 or 8 warps take a token: a lane holds
// a 16-byte chunk of dout and goes over the token's K rows with it, all K
// loads in flight, keeping a partial dot product for each; the warp, then
// the token's warps in order, join them.  Many tokens: a warp each, so that no
// barrier stands in the way; few: more warps a token.  Blocks past the
// tokens' zero the groups' padding rows.
// Measured (GB300, copy rate 6.68 TB/s): 131072 rows of 7168, 664 us, 6.0 TB/s
// (a block a token, whose threads met at two barriers: 874 us).
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
    int token_blocks, warps_per_token;
    uint16_t* dy;
    float* dw;
};

constexpr int kMaxK = 32;
constexpr int kWarps = 8;

template <int KT>  // K at compile time, or 0 for any K <= 32 (four rows at a time)
__global__ void __launch_bounds__(32 * kWarps, 3) combine_grad_kernel(const CombineGradArgs a) {
    __shared__ float sums[kWarps][kMaxK];
    pdl_wait();
    pdl_trigger();
    // Decided by the block as a whole: another block may record an error between
    // two warps' reads, and a token's warps meet at barriers below.
    if (__syncthreads_or(ld_volatile_s32(a.status) != 0)) return;
    const int64_t H = a.H;
    const int nvec = a.H / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (static_cast<int>(blockIdx.x) >= a.token_blocks) {  // zero one expert's padding rows
        const int e = static_cast<int>(blockIdx.x) - a.token_blocks;
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
    const int K = KT > 0 ? KT : a.K;
    constexpr int KB = KT > 0 ? KT : 4;
    const int per_block = kWarps / a.warps_per_token;
    const int part = warp % a.warps_per_token;
    // every warp of a block makes the same number of rounds (they may meet at a barrier)
    const int64_t stride = static_cast<int64_t>(a.token_blocks) * per_block;
    for (int64_t s0 = static_cast<int64_t>(blockIdx.x) * per_block; s0 < a.N; s0 += stride) {
        const int64_t s = s0 + warp / a.warps_per_token;
        bool live = s < a.N;
        int32_t my_raw = 0;
        float my_w = 0.f;
        bool bad = false;
        if (live && lane < K) {
            my_raw = raw_slot(__ldg(a.dst + s * K + lane));
            my_w = __ldg(a.w + s * K + lane);
            bad = my_raw < 0 || static_cast<int64_t>(my_raw) >= a.rows;
        }
        if (__any_sync(FULL_MASK, bad)) {
            if (bad) record_error(a.status, MOE_ERR_DEVICE_INDEX, my_raw);
            live = false;
        }
        float total = 0.f;  // lane k: this warp's part of dw[s][k]
        for (int k0 = 0; k0 < K && live; k0 += KB) {
            int64_t row[KB];
            float w[KB], dot[KB];
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                dot[k] = 0.f;
                row[k] = __shfl_sync(FULL_MASK, my_raw, (k0 + k) & 31) * H;
                w[k] = __shfl_sync(FULL_MASK, my_w, (k0 + k) & 31);
            }
            for (int c = part * 32 + lane; c < nvec; c += a.warps_per_token * 32) {
                float d[8];
                const uint4 dv = ld_stream_v4(a.dout + s * H + 8 * static_cast<int64_t>(c));
                uint4 v[KB];
#pragma unroll
                for (int k = 0; k < KB; ++k)
                    if (k0 + k < K) v[k] = ld_stream_v4(a.y + row[k] + 8 * static_cast<int64_t>(c));
                unpack8(dv, d);
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
            for (int k = 0; k < KB; ++k) {
                const float t = warp_sum(dot[k]);
                if (lane == k0 + k) total = t;
            }
        }
        if (a.warps_per_token == 1) {
            if (live && lane < K) a.dw[s * K + lane] = total;
        } else {
            __syncthreads();  // the last round's sums have been read
            sums[warp][lane] = total;
            __syncthreads();
            if (live && part == 0 && lane < K) {
                for (int i = 1; i < a.warps_per_token; ++i) total += sums[warp + i][lane];
                a.dw[s * K + lane] = total;
            }
        }
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
    if (N == 0) return MOE_OK;
    moe::CombineGradArgs a = {dout, y, topk_w, plan->dst, plan->zero_fill_ranges, plan->status, N, K, H, E, rows,
                              0,    0, dy,     dw};
    // a warp a token once that gives every SM its 16 warps, else more warps a token
    const int64_t sms = moe_host::num_sms();
    a.warps_per_token = 1;
    while (a.warps_per_token < moe::kWarps && static_cast<int64_t>(N) * a.warps_per_token < sms * 16) a.warps_per_token *= 2;
    const int per_block = moe::kWarps / a.warps_per_token;
    const int64_t blocks = (static_cast<int64_t>(N) + per_block - 1) / per_block;
    a.token_blocks = static_cast<int>(blocks < sms * 16 ? blocks : sms * 16);
    const dim3 grid(static_cast<unsigned>(a.token_blocks + E)), block(32 * moe::kWarps);
    switch (K) {
        case 1: return moe_host::launch(moe::combine_grad_kernel<1>, grid, block, 0, stream, a);
        case 2: return moe_host::launch(moe::combine_grad_kernel<2>, grid, block, 0, stream, a);
        case 4: return moe_host::launch(moe::combine_grad_kernel<4>, grid, block, 0, stream, a);
        case 8: return moe_host::launch(moe::combine_grad_kernel<8>, grid, block, 0, stream, a);
        default: return moe_host::launch(moe::combine_grad_kernel<0>, grid, block, 0, stream, a);
    }
}
