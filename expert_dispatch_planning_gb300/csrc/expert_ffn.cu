// expert_ffn.cu -- the experts' gated feed-forward over a plan's rows and
// its gradients (sm_103a).
//
// Five products, all grouped by expert (sum over k):
//   gated   g, u [row, i] = x[row, k] * w_gate_up[e][0|1][i][k]
//   down    y    [row, j] = h[row, k] * w_down[e][j][k]
//   dgate   dh   [row, i] = dy[row, k] * w_down[e][k][i]
//   dx      dx   [row, j] = dgate_up[row, k] * w_gate_up[e][k][j]
//   dw      dW[e][i][j]   = sum over the group's rows of left[row, i] * right[row, j]
// Plain shared-memory tiles of 64 x 64 with fp32 multiply-adds.
#include <cuda_fp8.h>

#include "vec8.cuh"

namespace moe {

enum Product { kGated, kDown, kDgate, kDx, kDw };

struct FfnArgs {
    const void* a;        // rows of the left operand
    const void* b;        // weights, or (kDw) the right operand's rows
    const float* a_scale;
    const float* b_scale;
    const float* preact_in;
    const int32_t* cu;
    const int32_t* count;
    int32_t* status;
    int64_t rows;
    int E, M, N, K;       // output width N, contraction length K (kDw: output M x N)
    uint16_t* out;
    float* preact_out;
};

template <typename T>
__device__ __forceinline__ float elem(const T* p, int64_t i);
template <>
__device__ __forceinline__ float elem(const uint16_t* p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}
template <>
__device__ __forceinline__ float elem(const uint8_t* p, int64_t i) {
    __nv_fp8_e4m3 v;
    v.__x = p[i];
    return static_cast<float>(v);
}
__device__ __forceinline__ uint16_t to_bf16(float v) { return static_cast<uint16_t>(pack2(v, 0.f) & 0xffffu); }

// A group's first row and row count; false (and an error) if it leaves [0, rows).
__device__ __forceinline__ bool group_of(const FfnArgs& a, int e, int64_t& first, int64_t& count, int64_t& padded) {
    first = __ldg(a.cu + e);
    count = __ldg(a.count + e);
    padded = static_cast<int64_t>(__ldg(a.cu + e + 1)) - first;
    if (count == 0) padded = 0;
    if (count < 0 || first < 0 || first + count > a.rows || padded < count || first + padded > a.rows) {
        record_error(a.status, MOE_ERR_DEVICE_INDEX, e);
        count = padded = 0;
        return false;
    }
    return true;
}

template <int P, typename T>
__global__ void __launch_bounds__(256) ffn_kernel(const FfnArgs a) {
    __shared__ float sa[16][65], sb[16][65], sb2[16][65];
    pdl_wait();
    pdl_trigger();
    if (ld_volatile_s32(a.status) != 0) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int n0 = blockIdx.x * 64;
    int e = 0;
    int64_t first = 0, count = 0, padded = 0, m0 = 0;
    if (P == kDw) {
        e = blockIdx.z;
        group_of(a, e, first, count, padded);
        m0 = static_cast<int64_t>(blockIdx.y) * 64;
    } else {
        int64_t t = blockIdx.y;
        for (e = 0; e < a.E; ++e) {
            group_of(a, e, first, count, padded);
            const int64_t tiles = (padded + 63) / 64;
            if (t < tiles) break;
            t -= tiles;
        }
        if (e == a.E) return;
        m0 = t * 64;
    }
    const int64_t kn = P == kDw ? count : a.K;
    const T* A = static_cast<const T*>(a.a);
    const T* B = static_cast<const T*>(a.b);
    float acc[4][4] = {}, acc2[4][4] = {};
    for (int64_t k0 = 0; k0 < kn; k0 += 16) {
        for (int i = tid; i < 1024; i += 256) {
            {   // left operand
                const int k = P == kDw ? i >> 6 : i & 15, m = P == kDw ? i & 63 : i >> 4;
                float v = 0.f;
                if (k0 + k < kn) {
                    if (P == kDw) {
                        if (m0 + m < a.M) v = elem(A, (first + k0 + k) * a.M + m0 + m);
                    } else if (m0 + m < count) {
                        v = elem(A, (first + m0 + m) * a.K + k0 + k);
                    }
                }
                sa[k][m] = v;
            }
            const bool row_k = P == kGated || P == kDown;  // k is the weights' contiguous index
            const int k = row_k ? i & 15 : i >> 6, n = row_k ? i >> 4 : i & 63;
            float v = 0.f, v2 = 0.f;
            if (k0 + k < kn && n0 + n < a.N) {
                if (P == kGated) {
                    const int64_t at = (static_cast<int64_t>(e) * 2 * a.N + n0 + n) * a.K + k0 + k;
                    v = elem(B, at);
                    v2 = elem(B, at + static_cast<int64_t>(a.N) * a.K);
                } else if (P == kDown) {
                    v = elem(B, (static_cast<int64_t>(e) * a.N + n0 + n) * a.K + k0 + k);
                } else if (P == kDw) {
                    v = elem(B, (first + k0 + k) * a.N + n0 + n);
                } else {
                    v = elem(B, (static_cast<int64_t>(e) * a.K + k0 + k) * a.N + n0 + n);
                }
            }
            sb[k][n] = v;
            if (P == kGated) sb2[k][n] = v2;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
                    if (P == kGated) acc2[i][j] = fmaf(sa[k][ty + 16 * i], sb2[k][tx + 16 * j], acc2[i][j]);
                }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i;
            const int n = n0 + tx + 16 * j;
            if (n >= a.N) continue;
            if (P == kDw) {
                if (m < a.M) a.out[(static_cast<int64_t>(e) * a.M + m) * a.N + n] = to_bf16(acc[i][j]);
                continue;
            }
            const int64_t row = first + m;
            if (m >= count) {  // the group's padding
                if (m < padded && (P == kDown || P == kDx)) a.out[row * a.N + n] = 0;
                continue;
            }
            if (P == kGated) {
                float g = acc[i][j], u = acc2[i][j];
                if (a.a_scale != nullptr) {
                    g *= a.a_scale[row] * a.b_scale[static_cast<int64_t>(e) * 2 * a.N + n];
                    u *= a.a_scale[row] * a.b_scale[(static_cast<int64_t>(e) * 2 + 1) * a.N + n];
                }
                if (a.preact_out != nullptr) {
                    a.preact_out[row * 2 * a.N + n] = g;
                    a.preact_out[row * 2 * a.N + a.N + n] = u;
                }
                a.out[row * a.N + n] = to_bf16(g / (1.f + expf(-g)) * u);
            } else if (P == kDgate) {
                const float g = a.preact_in[row * 2 * a.N + n], u = a.preact_in[row * 2 * a.N + a.N + n];
                const float sig = 1.f / (1.f + expf(-g));
                a.out[row * 2 * a.N + n] = to_bf16(acc[i][j] * u * sig * (1.f + g * (1.f - sig)));
                a.out[row * 2 * a.N + a.N + n] = to_bf16(acc[i][j] * g * sig);
            } else {
                a.out[row * a.N + n] = to_bf16(acc[i][j]);
            }
        }
}

}  // namespace moe

// ---------------------------------------------------------------- host
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_sizes(int64_t rows, int E, int H, int I, const MoePlanOut* plan) {
    if (plan == nullptr || plan->cu_seqlens == nullptr || plan->tokens_per_expert == nullptr || plan->status == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (rows < 0 || rows >= (int64_t(1) << 31) || E < 1 || E > 1024 || H < 8 || H % 8 != 0 || H >= (1 << 20) || I < 8 ||
        I % 8 != 0 || I >= (1 << 20))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

template <int P, typename T>
int launch_product(const moe::FfnArgs& a, cudaStream_t stream) {
    const int64_t m_tiles = P == moe::kDw ? (a.M + 63) / 64 : (a.rows + 63) / 64 + a.E;
    const dim3 grid(static_cast<unsigned>((a.N + 63) / 64), static_cast<unsigned>(m_tiles), P == moe::kDw ? a.E : 1);
    return moe_host::launch(moe::ffn_kernel<P, T>, grid, dim3(256), 0, stream, a);
}

}  // namespace

extern "C" MOE_API int moe_expert_ffn(const void* x, const float* x_scale, const void* w_gate_up, const float* w_scale,
                                      const uint16_t* w_down, int64_t rows, int E, int H, int I, int x_dtype,
                                      const MoePlanOut* plan, uint16_t* h, float* preact, uint16_t* y,
                                      cudaStream_t stream) {
    const int rc = check_sizes(rows, E, H, I, plan);
    if (rc != MOE_OK) return rc;
    if (x_dtype != MOE_DTYPE_BF16 && x_dtype != MOE_DTYPE_E4M3) return MOE_ERR_INVALID_ARG;
    const bool fp8 = x_dtype == MOE_DTYPE_E4M3;
    if (fp8 && H % 16 != 0) return MOE_ERR_INVALID_ARG;
    if (w_gate_up == nullptr || w_down == nullptr || fp8 != (w_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (x == nullptr || h == nullptr || y == nullptr || fp8 != (x_scale != nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(h) || !aligned16(preact) ||
        !aligned16(y) || !aligned16(x_scale) || !aligned16(w_scale))
        return MOE_ERR_INVALID_ARG;
    if (fp8 && preact != nullptr) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    moe::FfnArgs a = {};
    a.cu = plan->cu_seqlens;
    a.count = plan->tokens_per_expert;
    a.status = plan->status;
    a.rows = rows;
    a.E = E;
    a.a = x;
    a.b = w_gate_up;
    a.a_scale = x_scale;
    a.b_scale = w_scale;
    a.N = I;
    a.K = H;
    a.out = h;
    a.preact_out = preact;
    const int rg = fp8 ? launch_product<moe::kGated, uint8_t>(a, stream) : launch_product<moe::kGated, uint16_t>(a, stream);
    if (rg != MOE_OK) return rg;
    a.a = h;
    a.b = w_down;
    a.a_scale = a.b_scale = nullptr;
    a.N = H;
    a.K = I;
    a.out = y;
    return launch_product<moe::kDown, uint16_t>(a, stream);
}

extern "C" MOE_API int moe_expert_ffn_backward(const uint16_t* dy, const uint16_t* x, const uint16_t* h,
                                               const float* preact, const uint16_t* w_gate_up, const uint16_t* w_down,
                                               int64_t rows, int E, int H, int I, const MoePlanOut* plan,
                                               uint16_t* dgate_up, uint16_t* dx, uint16_t* dw_gate_up,
                                               uint16_t* dw_down, cudaStream_t stream) {
    int rc = check_sizes(rows, E, H, I, plan);
    if (rc != MOE_OK) return rc;
    if (w_gate_up == nullptr || w_down == nullptr) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (dy == nullptr || x == nullptr || h == nullptr || preact == nullptr || dgate_up == nullptr))
        return MOE_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(dy), static_cast<const void*>(x), static_cast<const void*>(h),
                          static_cast<const void*>(preact), static_cast<const void*>(w_gate_up),
                          static_cast<const void*>(w_down), static_cast<const void*>(dgate_up),
                          static_cast<const void*>(dx), static_cast<const void*>(dw_gate_up),
                          static_cast<const void*>(dw_down)})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) {
        const size_t bytes = static_cast<size_t>(E) * H * I * sizeof(uint16_t);
        if (dw_gate_up != nullptr && cudaMemsetAsync(dw_gate_up, 0, 2 * bytes, stream) != cudaSuccess)
            return MOE_ERR_CUDA;
        if (dw_down != nullptr && cudaMemsetAsync(dw_down, 0, bytes, stream) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    moe::FfnArgs a = {};
    a.cu = plan->cu_seqlens;
    a.count = plan->tokens_per_expert;
    a.status = plan->status;
    a.rows = rows;
    a.E = E;
    if (dx != nullptr || dw_gate_up != nullptr) {
        a.a = dy;
        a.b = w_down;
        a.preact_in = preact;
        a.N = I;
        a.K = H;
        a.out = dgate_up;
        rc = launch_product<moe::kDgate, uint16_t>(a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dx != nullptr) {
        a.a = dgate_up;
        a.b = w_gate_up;
        a.N = H;
        a.K = 2 * I;
        a.out = dx;
        rc = launch_product<moe::kDx, uint16_t>(a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dw_gate_up != nullptr) {
        a.a = dgate_up;
        a.b = x;
        a.M = 2 * I;
        a.N = H;
        a.out = dw_gate_up;
        rc = launch_product<moe::kDw, uint16_t>(a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dw_down != nullptr) {
        a.a = dy;
        a.b = h;
        a.M = H;
        a.N = I;
        a.out = dw_down;
        rc = launch_product<moe::kDw, uint16_t>(a, stream);
    }
    return rc;
}
