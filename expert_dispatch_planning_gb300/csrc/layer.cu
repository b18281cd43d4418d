// layer.cu -- a whole mixture-of-experts layer for a few tokens (sm_103a).
//
// For N <= 64 tokens: the router's choice, and for every chosen pair (s, k)
// with e = idx[s][k]
//   g = x[s] . w_gate[e]^T,  u = x[s] . w_up[e]^T,  h = bf16(silu(g) * u),
//   out[s] = bf16(sum over k of w[s][k] * (h . w_down[e]^T)).
// A decoding step reads the weights of every chosen expert for a handful of
// rows: that is all it takes time for.  So nothing is permuted or padded; the
// weights stream from memory once, straight into the registers that the matrix
// instruction takes them from, and everything else hides behind them.
//
// Three launches: moe_route_topk, gate/up, down.  Each block of the second and
// third finds the chosen experts and their tokens by itself from topk_idx (a
// 64-bit set of tokens for every expert).
//
// Products.  mma.m16n8k16 with 16 weight rows as its M side and up to 8 tokens
// as its N side: an expert has a few tokens, and a tcgen05 tile of 64 or 128
// rows would leave most SMs without one.  A lane's place in the fragment wants
// 2 + 2 elements of a row for every 16 of k; since a sum may be taken in any
// order of k, as long as both operands agree, a lane takes 16 contiguous bytes
// of its row (and of its token's) instead: four lanes read 64 bytes of a row,
// without shared memory or shuffles.  8-bit operands become fp16 in registers
// (exact), their products are exact in the fp32 accumulator.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>

#include "vec8.cuh"

namespace moe {

constexpr int kLayerThreads = 256;
constexpr int kLayerWarps = kLayerThreads / 32;

struct LayerArgs {
    const void* x;
    const float* x_scale;
    const void* w_gate_up;
    const float* w_scale;
    const uint16_t* w_down;
    const int32_t* topk_idx;
    const float* topk_w;
    uint16_t* h;  // [N*K][I], rows in the order of experts, then tokens
    uint16_t* out;
    int N, K, E, H, I;
};

// ---------------------------------------------------------------- the chosen experts
// In shared memory: expert[a] and begin[a] of the a-th chosen expert (begin[count]
// = pairs), and for every place its token and weight.  All threads of the block call.
struct Chosen {
    unsigned long long* tokens;  // [E] sets of tokens
    int* expert;                 // [slots]
    int* begin;                  // [slots + 1]
    int* sums;                   // [warps + 1] of the scan
    float* weight;               // [N*K]
    uint8_t* token;              // [N*K]
    int count;

    static __host__ __device__ int slots(int N, int K, int E) { return N * K < E ? N * K : E; }
    static __host__ __device__ size_t bytes(int N, int K, int E) {
        const size_t s = 8 * static_cast<size_t>(E) + 4 * (2 * slots(N, K, E) + 1) + 4 * (kLayerWarps + 1) + 5 * N * K;
        return (s + 15) / 16 * 16;
    }
    __device__ Chosen(uint8_t* smem, const LayerArgs& a) {
        const int n = slots(a.N, a.K, a.E);
        tokens = reinterpret_cast<unsigned long long*>(smem);
        expert = reinterpret_cast<int*>(tokens + a.E);
        begin = expert + n;
        sums = begin + n + 1;
        weight = reinterpret_cast<float*>(sums + kLayerWarps + 1);
        token = reinterpret_cast<uint8_t*>(weight + a.N * a.K);
    }
    __device__ int size(int i) const { return begin[i + 1] - begin[i]; }

    __device__ void find(const LayerArgs& a) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pairs = a.N * a.K;
        for (int e = tid; e < a.E; e += kLayerThreads) tokens[e] = 0;
        __syncthreads();
        for (int f = tid; f < pairs; f += kLayerThreads) {
            const int e = a.topk_idx[f];
            if (static_cast<unsigned>(e) < static_cast<unsigned>(a.E)) atomicOr(&tokens[e], 1ull << (f / a.K));
        }
        __syncthreads();
        // a thread has a run of experts: counts of chosen ones and of pairs before it, in one word
        const int per = (a.E + kLayerThreads - 1) / kLayerThreads, e0 = tid * per;
        int mine = 0;
        for (int e = e0; e < e0 + per && e < a.E; ++e)
            if (tokens[e] != 0) mine += 0x10000 + __popcll(tokens[e]);
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(FULL_MASK, before, o);
            if (lane >= o) before += t;
        }
        if (lane == 31) sums[warp] = before;
        __syncthreads();
        int all = 0;
        before -= mine;
#pragma unroll
        for (int w = 0; w < kLayerWarps; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        count = all >> 16;
        int place = before >> 16, at = before & 0xffff;
        for (int e = e0; e < e0 + per && e < a.E; ++e) {
            if (tokens[e] == 0) continue;
            expert[place] = e;
            begin[place] = at;
            ++place;
            at += __popcll(tokens[e]);
        }
        if (tid == 0) begin[count] = all & 0xffff;
        __syncthreads();
        for (int i = warp; i < count; i += kLayerWarps) {  // a warp an expert, a lane a token (and its 32nd next)
            const unsigned long long set = tokens[expert[i]];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int s = lane + 32 * half;
                if (s < a.N && (set >> s & 1) != 0) {
                    const int p = begin[i] + __popcll(set & ((1ull << s) - 1));
                    token[p] = static_cast<uint8_t>(s);
                    float w = 0.f;
                    for (int k = 0; k < a.K; ++k)
                        if (a.topk_idx[s * a.K + k] == expert[i]) w = a.topk_w[s * a.K + k];
                    weight[p] = w;
                }
            }
        }
        __syncthreads();
    }
};

// ---------------------------------------------------------------- products
// Sixteen bytes of a row as the matrix instruction's words: eight bf16, or
// sixteen e4m3 as fp16.
template <bool Q>
struct Fragment {
    uint32_t w[Q ? 8 : 4];
    __device__ __forceinline__ explicit Fragment(const uint4& v) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Q) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                        static_cast<__nv_fp8x2_storage_t>(j == 0 ? u[i] & 0xffffu : u[i] >> 16), __NV_E4M3);
                    w[2 * i + j] = h.x | static_cast<uint32_t>(h.y) << 16;
                }
            } else {
                w[i] = u[i];
            }
        }
    }
};

template <bool Q>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (Q) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
}

// c += rows (lo: row g, hi: row g + 8 of the lane's sixteen) times tokens.
template <bool Q>
__device__ __forceinline__ void product(float (&c)[4], const Fragment<Q>& lo, const Fragment<Q>& hi,
                                        const Fragment<Q>& b) {
#pragma unroll
    for (int i = 0; i < (Q ? 4 : 2); ++i) mma<Q>(c, lo.w[2 * i], hi.w[2 * i], lo.w[2 * i + 1], hi.w[2 * i + 1], b.w[2 * i], b.w[2 * i + 1]);
}

// Not a read-only load: h comes from the launch before, which may still run as this one starts.
__device__ __forceinline__ uint4 load16(const uint8_t* p, bool inside) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (inside)
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint4 stream16(const uint8_t* p, bool inside) {
    return inside ? ld_stream_v4(p) : make_uint4(0, 0, 0, 0);
}

// acc += rows times tokens over the lane's 16-byte blocks first .. last of k
// (64 bytes of a row each).  lo, hi: the lane's two weight rows, null where there is
// none; col[j]: its token's row in the j-th eight, null where there is none.
// bytes: a row's length.
template <bool Q, int NT>
__device__ __forceinline__ void stream_rows(float (&acc)[NT][4], const uint8_t* lo, const uint8_t* hi,
                                            const uint8_t* const (&col)[NT], int first, int last, int bytes, int t) {
    constexpr int U = 4;  // blocks asked for at a time
    for (int b = first; b < last; b += U) {
        uint4 wl[U], wh[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int at = (b + i) * 64 + t * 16;
            const bool in = b + i < last && at < bytes;
            wl[i] = stream16(lo + at, in && lo != nullptr);
            wh[i] = stream16(hi + at, in && hi != nullptr);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int at = (b + i) * 64 + t * 16;
            const bool in = b + i < last && at < bytes;
            uint4 xs[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) xs[j] = load16(col[j] + at, in && col[j] != nullptr);
            const Fragment<Q> fl(wl[i]), fh(wh[i]);
#pragma unroll
            for (int j = 0; j < NT; ++j) product<Q>(acc[j], fl, fh, Fragment<Q>(xs[j]));
        }
    }
}

// ---------------------------------------------------------------- gate and up
__device__ __forceinline__ float silu(float g) {
    const float e = expf(-fabsf(g));
    return g * __fdiv_rn(g >= 0.f ? 1.f : e, 1.f + e);
}

// Up to eight channels of one expert: gate rows as the instruction's first
// eight rows, up rows as its others, so that a lane ends with both; the block's warps
// share k.  `sum`: [warps][NT][32] float4.
template <bool Q, int NT>
__device__ __forceinline__ void gate_up_tile(const LayerArgs& a, const Chosen& c, float4* sum, int i, int channel,
                                             int channels) {
    constexpr int kSize = Q ? 1 : 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int e = c.expert[i], first_pair = c.begin[i], cols = c.begin[i + 1] - first_pair;
    const int64_t row_bytes = static_cast<int64_t>(a.H) * kSize;
    const uint8_t* w = static_cast<const uint8_t*>(a.w_gate_up);
    const uint8_t *lo = nullptr, *hi = nullptr;
    if (g < channels) {
        const int64_t r = (static_cast<int64_t>(e) * 2 * a.I + channel + g) * row_bytes;
        lo = w + r;
        hi = w + r + a.I * row_bytes;
    }
    const uint8_t* col[NT];
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int p = 8 * j + g;
        col[j] = p < cols ? static_cast<const uint8_t*>(a.x) + c.token[first_pair + p] * row_bytes : nullptr;
        acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    }
    const int bytes = static_cast<int>(row_bytes), blocks = (bytes + 63) / 64;
    stream_rows<Q, NT>(acc, lo, hi, col, warp * blocks / kLayerWarps, (warp + 1) * blocks / kLayerWarps, bytes, t);
#pragma unroll
    for (int j = 0; j < NT; ++j) sum[(warp * NT + j) * 32 + lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    __syncthreads();
    for (int v = threadIdx.x; v < NT * 32; v += kLayerThreads) {
        float4 s = sum[v];
#pragma unroll
        for (int k = 1; k < kLayerWarps; ++k) {
            const float4 o = sum[k * NT * 32 + v];
            s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
        }
        const int row = (v & 31) >> 2, p = 8 * (v >> 5) + 2 * (v & 3);
        if (row < channels) {
            const int ch = channel + row;
            float wg = 1.f, wu = 1.f;
            if constexpr (Q) {
                wg = __ldg(a.w_scale + static_cast<int64_t>(e) * 2 * a.I + ch);
                wu = __ldg(a.w_scale + static_cast<int64_t>(e) * 2 * a.I + a.I + ch);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (p + j >= cols) continue;
                float gate = j == 0 ? s.x : s.y, up = j == 0 ? s.z : s.w;
                if constexpr (Q) {
                    const float xs = __ldg(a.x_scale + c.token[first_pair + p + j]);
                    gate = gate * wg * xs;
                    up = up * wu * xs;
                }
                const __nv_bfloat16 h = __float2bfloat16_rn(silu(gate) * up);
                a.h[static_cast<int64_t>(first_pair + p + j) * a.I + ch] = __bfloat16_as_ushort(h);
            }
        }
    }
    __syncthreads();
}

// MAXT: eights of tokens an expert can have.
template <bool Q, int MAXT>
__global__ void __launch_bounds__(kLayerThreads) layer_gate_up_kernel(const LayerArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    float4* sum = reinterpret_cast<float4*>(smem);
    Chosen c(smem + sizeof(float4) * kLayerWarps * MAXT * 32, a);
    pdl_wait();
    pdl_trigger();
    c.find(a);
    // every block takes an equal run of the chosen experts' channels
    const int64_t all = static_cast<int64_t>(c.count) * a.I;
    int64_t at = blockIdx.x * all / gridDim.x;
    const int64_t end = (blockIdx.x + 1) * all / gridDim.x;
    while (at < end) {
        const int i = static_cast<int>(at / a.I), channel = static_cast<int>(at - static_cast<int64_t>(i) * a.I);
        int n = a.I - channel < 8 ? a.I - channel : 8;
        if (end - at < n) n = static_cast<int>(end - at);
        const int eights = (c.size(i) + 7) / 8;
        if (MAXT >= 8 && eights > 4) gate_up_tile<Q, MAXT >= 8 ? 8 : 1>(a, c, sum, i, channel, n);
        else if (MAXT >= 4 && eights > 2) gate_up_tile<Q, MAXT >= 4 ? 4 : 1>(a, c, sum, i, channel, n);
        else if (MAXT >= 2 && eights > 1) gate_up_tile<Q, MAXT >= 2 ? 2 : 1>(a, c, sum, i, channel, n);
        else gate_up_tile<Q, 1>(a, c, sum, i, channel, n);
        at += n;
    }
}

// ---------------------------------------------------------------- down
// Rows `first_row` .. of out for one expert's tokens, over blocks first .. last of k: added,
// weighted, to the warp's sums [ROWS][N].
template <int ROWS, int NT>
__device__ __forceinline__ void down_part(const LayerArgs& a, const Chosen& c, float* sum, int i, int first_row, int rows,
                                          int first, int last) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int first_pair = c.begin[i], cols = c.begin[i + 1] - first_pair;
    const int64_t row_bytes = static_cast<int64_t>(a.I) * 2;
    const uint8_t* w = reinterpret_cast<const uint8_t*>(a.w_down) +
                       (static_cast<int64_t>(c.expert[i]) * a.H + first_row) * row_bytes;
    const uint8_t* lo = g < rows ? w + g * row_bytes : nullptr;
    const uint8_t* hi = ROWS == 16 && g + 8 < rows ? w + (g + 8) * row_bytes : nullptr;
    const uint8_t* col[NT];
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int p = 8 * j + g;
        col[j] = p < cols ? reinterpret_cast<const uint8_t*>(a.h) + (first_pair + p) * row_bytes : nullptr;
        acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    }
    stream_rows<false, NT>(acc, lo, hi, col, first, last, static_cast<int>(row_bytes), t);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int p = 8 * j + 2 * t + (v & 1), row = g + (v >> 1) * 8;
            if (p < cols && row < ROWS) {
                float* s = sum + row * a.N + c.token[first_pair + p];
                *s = fmaf(c.weight[first_pair + p], acc[j][v], *s);
            }
        }
    __syncwarp();  // the next expert's tokens are other lanes'
}

// A block has ROWS rows of the output, its warps share the chosen experts' k.
template <int ROWS, int MAXT>
__global__ void __launch_bounds__(kLayerThreads) layer_down_kernel(const LayerArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem);  // [warps][ROWS][N]
    Chosen c(smem + sizeof(float) * kLayerWarps * ROWS * a.N, a);
    const int tid = threadIdx.x, warp = tid >> 5;
    for (int v = tid; v < kLayerWarps * ROWS * a.N; v += kLayerThreads) sums[v] = 0.f;
    c.find(a);
    pdl_wait();
    pdl_trigger();
    const int first_row = blockIdx.x * ROWS;
    const int rows = a.H - first_row < ROWS ? a.H - first_row : ROWS;
    const int blocks = (2 * a.I + 63) / 64;
    const int all = c.count * blocks;
    int at = static_cast<int>(static_cast<int64_t>(warp) * all / kLayerWarps);
    const int end = static_cast<int>(static_cast<int64_t>(warp + 1) * all / kLayerWarps);
    float* sum = sums + warp * ROWS * a.N;
    while (at < end) {
        const int i = at / blocks, first = at - i * blocks;
        const int last = end - at < blocks - first ? first + end - at : blocks;
        const int eights = (c.size(i) + 7) / 8;
        if (MAXT >= 8 && eights > 4) down_part<ROWS, MAXT >= 8 ? 8 : 1>(a, c, sum, i, first_row, rows, first, last);
        else if (MAXT >= 4 && eights > 2) down_part<ROWS, MAXT >= 4 ? 4 : 1>(a, c, sum, i, first_row, rows, first, last);
        else if (MAXT >= 2 && eights > 1) down_part<ROWS, MAXT >= 2 ? 2 : 1>(a, c, sum, i, first_row, rows, first, last);
        else down_part<ROWS, 1>(a, c, sum, i, first_row, rows, first, last);
        at += last - first;
    }
    __syncthreads();
    for (int v = tid; v < ROWS * a.N; v += kLayerThreads) {
        const int row = v % ROWS, s = v / ROWS;  // neighbouring threads write neighbouring elements
        if (row < rows) {
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < kLayerWarps; ++w) o += sums[(w * ROWS + row) * a.N + s];
            a.out[static_cast<int64_t>(s) * a.H + first_row + row] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
        }
    }
}

}  // namespace moe

// ---------------------------------------------------------------- host
namespace {

using namespace moe_host;
using moe::LayerArgs;

template <bool Q, int MAXT>
int launch_gate_up(const LayerArgs& a, cudaStream_t stream) {
    const size_t smem = sizeof(float4) * moe::kLayerWarps * MAXT * 32 + moe::Chosen::bytes(a.N, a.K, a.E);
    if (cudaFuncSetAttribute(moe::layer_gate_up_kernel<Q, MAXT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    return launch(moe::layer_gate_up_kernel<Q, MAXT>, dim3(static_cast<unsigned>(3 * num_sms())), dim3(moe::kLayerThreads),
                  smem, stream, a);
}

template <int ROWS, int MAXT>
int launch_down(const LayerArgs& a, cudaStream_t stream) {
    const size_t smem = sizeof(float) * moe::kLayerWarps * ROWS * a.N + moe::Chosen::bytes(a.N, a.K, a.E);
    if (cudaFuncSetAttribute(moe::layer_down_kernel<ROWS, MAXT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    return launch(moe::layer_down_kernel<ROWS, MAXT>, dim3(static_cast<unsigned>((a.H + ROWS - 1) / ROWS)),
                  dim3(moe::kLayerThreads), smem, stream, a);
}

template <int MAXT>
int launch_layer(const LayerArgs& a, bool q, cudaStream_t stream) {
    const int rc = q ? launch_gate_up<true, MAXT>(a, stream) : launch_gate_up<false, MAXT>(a, stream);
    if (rc != MOE_OK) return rc;
    return a.H / 16 >= 2 * num_sms() ? launch_down<16, MAXT>(a, stream) : launch_down<8, MAXT>(a, stream);
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace

extern "C" MOE_API size_t moe_layer_workspace_size(int N, int K, int I) {
    if (N < 0 || N > MOE_LAYER_MAX_TOKENS || K < 1 || K > 32 || I < 8 || I % 8 != 0 || I >= 1 << 20) return 0;
    const size_t pairs = static_cast<size_t>(N > 0 ? N : 1) * K;
    return pairs * I * 2 + 2 * round16(pairs * 4);
}

extern "C" MOE_API int moe_layer(const void* x, const float* x_scale, const float* logits, const float* bias,
                                 const void* w_gate_up, const float* w_scale, const uint16_t* w_down, int N, int E, int H,
                                 int I, int K, int x_dtype, int scoring, int renormalize, int n_group, int topk_group,
                                 float routed_scaling, int32_t* topk_idx, float* topk_w, uint16_t* out, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    const bool q = x_dtype == MOE_DTYPE_E4M3;
    if (!q && x_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
    if (N < 0 || H < 8 || H % (q ? 16 : 8) != 0 || I < 8 || I % 8 != 0 || H >= 1 << 20 || I >= 1 << 20)
        return MOE_ERR_INVALID_ARG;
    if ((x_scale != nullptr || w_scale != nullptr) && !q) return MOE_ERR_INVALID_ARG;
    if (N > MOE_LAYER_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
    if (N > 0 && (x == nullptr || w_gate_up == nullptr || w_down == nullptr || out == nullptr || workspace == nullptr ||
                  (q && (x_scale == nullptr || w_scale == nullptr))))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w_gate_up, 16) || !aligned(w_down, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(x_scale, 4) || !aligned(w_scale, 4))
        return MOE_ERR_INVALID_ARG;
    if (N > 0 && K >= 1 && K <= 32) {
        if (workspace_bytes < moe_layer_workspace_size(N, K, I)) return MOE_ERR_CAPACITY;
        uint8_t* rest = static_cast<uint8_t*>(workspace) + static_cast<size_t>(N) * K * I * 2;
        if (topk_idx == nullptr) topk_idx = reinterpret_cast<int32_t*>(rest);
        if (topk_w == nullptr) topk_w = reinterpret_cast<float*>(rest + round16(static_cast<size_t>(N) * K * 4));
    }
    // the router's own checks of logits, bias, E, K and its options come with its call
    const int rc = moe_route_topk(logits, bias, N, E, K, scoring, renormalize, n_group, topk_group, routed_scaling, topk_idx,
                                  topk_w, stream);
    if (rc != MOE_OK || N == 0) return rc;
    const LayerArgs a = {x, x_scale, w_gate_up, w_scale, w_down, topk_idx, topk_w, static_cast<uint16_t*>(workspace), out,
                         N, K, E, H, I};
    if (N <= 8) return launch_layer<1>(a, q, stream);
    if (N <= 16) return launch_layer<2>(a, q, stream);
    if (N <= 32) return launch_layer<4>(a, q, stream);
    return launch_layer<8>(a, q, stream);
}
