// expert_ffn.cu -- the experts' gated feed-forward over a plan's rows and
// its gradients (sm_103a).
//
// Five products, all grouped by expert (sum over k):
//   gated   g, u [row, i] = x[row, k] * w_gate_up[e][0|1][i][k]
//   down    y    [row, j] = h[row, k] * w_down[e][j][k]
//   dgate   dh   [row, i] = dy[row, k] * w_down[e][k][i]
//   dx      dx   [row, j] = dgate_up[row, k] * w_gate_up[e][k][j]
//   dw      dW[e][i][j]   = sum over the group's rows of left[row, i] * right[row, j]
//
// One persistent kernel, one block an SM.  A tile is 128 rows of the output by
// up to 256 columns; its fp32 accumulators lie in tensor memory, twice, so
// that one tile's epilogue runs under the next one's products.  Warp 0 brings
// 128-byte wide slices of both operands into a ring of shared-memory stages
// (tensor copies, 128-byte swizzle), warp 1 issues the matrix instructions,
// warps 2-5 read the accumulators (32 rows each) and write the output.  The
// gated product has the gate's and the up projection's columns of the same
// channels side by side in one tile, so that silu(g) * u needs no exchange;
// dgate applies the activation's gradient to dh in its epilogue, so that dh
// is never written.
//
// Operands: where k is the contiguous index (x, h, dy, dgate_up; weights of
// gated and down) a stage holds rows of 64 k's (128 in 8 bits); where it is
// not (weights of dgate and dx, both of dw) a stage holds 64 rows of k, each
// with 64 of the tile's rows or columns, and the instruction reads it
// transposed.  Slices that leave an array are filled with zeros by the copy.
// In dw the last slice of a group runs on into other rows, which may hold
// anything: the issuing warp zeroes them in both operands first.
#include <cuda_fp8.h>

#include "tensor_core.cuh"
#include "vec8.cuh"

namespace moe {

enum Product { kGated, kDown, kDgate, kDx, kDw };

constexpr int kTileM = 128;
constexpr int kRing = 196 * 1024;  // bytes of shared memory for the stages
constexpr int kMaxStages = 16;
constexpr int kThreads = 192;
constexpr int kSlice = 128;        // bytes of k (or of a 64-element run) in a stage's row

struct FfnArgs {
    const float* a_scale;
    const float* b_scale;
    const float* preact_in;
    const int32_t* cu;
    const int32_t* count;
    int32_t* status;
    int64_t rows;
    int E, M, N, K;       // output width N, contraction length K (dw: output M x N)
    uint16_t* out;
    float* preact_out;
    int64_t timeout_ns;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int failed;
    int stop;             // the plan's status held an error
    int scan[kThreads / 32];
    int most[kThreads / 32];
};

struct Tile {
    int e;
    int64_t first;   // the group's first row
    int count;       // its rows
    int padded;      // and with its padding
    int m0, n0;      // the tile's first output row (within the group; dw: of M) and column
    int slices;      // of k
};

// What every warp of a block knows about the work.
struct Work {
    const int* first;
    const int* count;
    const int* padded;
    const int* prefix;  // row tiles before each expert (not dw)
    int E, M, N, k_slices;
    int cols;           // output columns of a tile
    int n_tiles;
    int64_t tiles;
};

template <int P>
__device__ __forceinline__ Tile locate(const Work& w, int64_t t) {
    Tile r;
    int mt;
    int64_t at;
    if constexpr (P == kDw) {
        mt = (w.M + kTileM - 1) / kTileM;
        const int64_t per = static_cast<int64_t>(mt) * w.n_tiles;
        r.e = static_cast<int>(t / per);
        at = t - r.e * per;
    } else {
        int lo = 0, hi = w.E;  // the expert with prefix[e] * n_tiles <= t < prefix[e + 1] * n_tiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (static_cast<int64_t>(w.prefix[mid]) * w.n_tiles <= t) lo = mid;
            else hi = mid;
        }
        r.e = lo;
        mt = w.prefix[lo + 1] - w.prefix[lo];
        at = t - static_cast<int64_t>(w.prefix[lo]) * w.n_tiles;
    }
    // bands of 16 row tiles, column by column: what the blocks work on at one time stays in L2
    constexpr int kBand = 16;
    const int band = static_cast<int>(at / (kBand * static_cast<int64_t>(w.n_tiles)));
    const int in_band = static_cast<int>(at - band * (kBand * static_cast<int64_t>(w.n_tiles)));
    const int height = min(kBand, mt - band * kBand);
    r.m0 = (band * kBand + in_band % height) * kTileM;
    r.n0 = in_band / height * w.cols;
    r.first = w.first[r.e];
    r.count = w.count[r.e];
    r.padded = w.padded[r.e];
    r.slices = P == kDw ? (r.count + 63) / 64 : w.k_slices;
    return r;
}

// Bounded wait; on a timeout the block gives up (`failed`) and the plan's status says so.
__device__ __forceinline__ bool wait(const FfnArgs& a, Shared* sh, uint64_t* bar, uint32_t parity) {
    if (mbar_wait_bounded(bar, parity, static_cast<uint64_t>(a.timeout_ns))) return true;
    *reinterpret_cast<volatile int*>(&sh->failed) = 1;
    record_error(a.status, MOE_ERR_DEVICE_TIMEOUT, blockIdx.x);
    return false;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) { return pack2(lo, hi); }

// silu(g) = g * sigmoid(g) and sigmoid(g).  The hardware exponential and
// division are within 2^-20 of the exact value for |g| < 16; beyond, where
// the sigmoid is 0 or 1 to bf16's precision or the result tiny, the relative
// error grows as |g| * 2^-24.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + __expf(-g)); }

// Eight columns of a row, as bf16.
__device__ __forceinline__ void store8_bf16(uint16_t* p, const float* v) {
    st_v4(p, make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])));
}

template <int P>
__device__ void epilogue(const FfnArgs& a, const Tile& t, int bn, uint32_t acc, int quarter, int lane, int thread) {
    const int cols = P == kGated ? bn / 2 : bn;
    const int m = t.m0 + quarter * 32 + lane;
    const bool live = P == kDw ? m < a.M : m < t.count;
    const bool any = P == kDw ? t.m0 + quarter * 32 < a.M : t.m0 + quarter * 32 < t.count;
    const int64_t N = a.N;
    const int64_t row = P == kDw ? static_cast<int64_t>(t.e) * a.M + m : t.first + m;
    const uint32_t lane_addr = acc + (static_cast<uint32_t>(quarter * 32) << 16);
    float row_scale = 1.f;
    if (P == kGated && a.a_scale != nullptr && live) row_scale = __ldg(a.a_scale + row);
    for (int c = 0; c < cols && any; c += 16) {
        const int n = t.n0 + c;
        if (n >= a.N) break;
        const int width = min(16, a.N - n);  // 8 or 16
        uint32_t v0[16], v1[16];
        float f[16];
        __syncwarp();  // the loads below are the whole warp's
        if (P == kDw && t.slices == 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v0[j] = 0u;
        } else {
            tmem_load16(lane_addr + c, v0);
            if constexpr (P == kGated) tmem_load16(lane_addr + cols + c, v1);
        }
        if constexpr (P == kDgate) {
            float g[16], u[16];
            if (live) {
                const float* pre = a.preact_in + row * 2 * N + n;
                for (int j = 0; j < width; j += 4) {
                    *reinterpret_cast<float4*>(g + j) = __ldg(reinterpret_cast<const float4*>(pre + j));
                    *reinterpret_cast<float4*>(u + j) = __ldg(reinterpret_cast<const float4*>(pre + N + j));
                }
            }
            tmem_wait_load();
            if (live) {
                float d[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float dh = __uint_as_float(v0[j]), s = sigmoid(g[j]);
                    f[j] = dh * u[j] * s * fmaf(g[j], 1.f - s, 1.f);
                    d[j] = dh * g[j] * s;
                }
                uint16_t* out = a.out + row * 2 * N + n;
                store8_bf16(out, f);
                store8_bf16(out + N, d);
                if (width == 16) {
                    store8_bf16(out + 8, f + 8);
                    store8_bf16(out + N + 8, d + 8);
                }
            }
            continue;
        }
        tmem_wait_load();
        if (!live) continue;
        if constexpr (P == kGated) {
            float g[16], u[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                g[j] = __uint_as_float(v0[j]);
                u[j] = __uint_as_float(v1[j]);
            }
            if (a.a_scale != nullptr) {
                const float* ws = a.b_scale + static_cast<int64_t>(t.e) * 2 * N + n;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < width) {
                        g[j] *= row_scale * __ldg(ws + j);
                        u[j] *= row_scale * __ldg(ws + N + j);
                    }
            }
            if (a.preact_out != nullptr) {
                float* pre = a.preact_out + row * 2 * N + n;
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    if (j < width) {
                        *reinterpret_cast<float4*>(pre + j) = make_float4(g[j], g[j + 1], g[j + 2], g[j + 3]);
                        *reinterpret_cast<float4*>(pre + N + j) = make_float4(u[j], u[j + 1], u[j + 2], u[j + 3]);
                    }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = silu(g[j]) * u[j];
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v0[j]);
        }
        store8_bf16(a.out + row * N + n, f);
        if (width == 16) store8_bf16(a.out + row * N + n + 8, f + 8);
    }
    if constexpr (P == kDown || P == kDx) {
        // the group's last row tile zeroes its padding, which may go on past the tile
        if (t.m0 + kTileM >= t.count && t.padded > t.count) {
            const int chunks = (min(cols, a.N - t.n0) + 7) / 8;
            const int64_t todo = static_cast<int64_t>(t.padded - t.count) * chunks;
            for (int64_t i = thread; i < todo; i += 128) {
                const int64_t r = t.first + t.count + i / chunks;
                st_v4(a.out + r * N + t.n0 + 8 * (i % chunks), make_uint4(0u, 0u, 0u, 0u));
            }
        }
    }
}

template <int P, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_a16,
               const __grid_constant__ CUtensorMap map_b, const FfnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    constexpr bool kAmn = P == kDw, kBmn = P == kDgate || P == kDx || P == kDw;  // k is not the contiguous index
    constexpr int kElems = FP8 ? 128 : 64;                                       // k's of a slice

    uint8_t* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Shared* sh = reinterpret_cast<Shared*>(ring + kRing);
    int* first = reinterpret_cast<int*>(sh + 1);
    int *count = first + a.E, *padded = count + a.E, *prefix = padded + a.E;  // prefix: E + 1

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        tensor_prefetch(&map_a);
        tensor_prefetch(&map_b);
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], 4);
        }
        fence_mbar_init();
        sh->failed = 0;
    }
    if (warp == 1) tmem_alloc(&sh->tmem, 512);
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh->stop = ld_volatile_s32(a.status) != 0;

    // ---- the groups: row tiles before each expert, and the longest group
    const int per = (a.E + kThreads - 1) / kThreads;
    int mine = 0, longest = 0;
    for (int e = tid * per; e < min(a.E, (tid + 1) * per); ++e) {
        const int64_t f = __ldg(a.cu + e), c = __ldg(a.count + e), p = c == 0 ? 0 : __ldg(a.cu + e + 1) - f;
        const bool fits = c >= 0 && f >= 0 && p >= c && f + p <= a.rows;
        if (!fits) record_error(a.status, MOE_ERR_DEVICE_INDEX, e);
        first[e] = fits ? static_cast<int>(f) : 0;
        count[e] = fits ? static_cast<int>(c) : 0;
        padded[e] = fits ? static_cast<int>(p) : 0;
        mine += (count[e] + kTileM - 1) / kTileM;
        longest = max(longest, count[e]);
    }
    int before = mine;  // inclusive over the warp, then exclusive over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, before, o);
        if (lane >= o) before += v;
    }
    longest = __reduce_max_sync(FULL_MASK, longest);
    if (lane == 31) sh->scan[warp] = before;
    if (lane == 0) sh->most[warp] = longest;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int row_tiles = 0;
    before -= mine;
    longest = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh->scan[w];
        row_tiles += sh->scan[w];
        longest = max(longest, sh->most[w]);
    }
    for (int e = tid * per; e < min(a.E, (tid + 1) * per); ++e) {
        prefix[e] = before;
        before += (count[e] + kTileM - 1) / kTileM;
    }
    if (tid == 0) prefix[a.E] = row_tiles;

    // ---- the tile's width: the fewest rounds of the grid, each weighed by its
    // columns and what a tile costs beside them (its rows' copies, its start)
    const int64_t m_tiles = P == kDw ? static_cast<int64_t>(a.E) * ((a.M + kTileM - 1) / kTileM) : row_tiles;
    const int a_rows = P == kDw || longest > 64 ? kTileM : max(16, (longest + 15) / 16 * 16);
    int bn = 256;
    int64_t best = -1;
    for (int b = 256; b >= 64; b >>= 1) {
        const int c = P == kGated ? b / 2 : b;
        const int64_t rounds = (m_tiles * ((a.N + c - 1) / c) + gridDim.x - 1) / gridDim.x;
        const int64_t cost = rounds * (b + a_rows / 4 + 16);
        if (best < 0 || cost < best) {
            best = cost;
            bn = b;
        }
    }
    const uint32_t a_bytes = static_cast<uint32_t>(a_rows) * kSlice;
    const uint32_t stage_bytes = a_bytes + static_cast<uint32_t>(bn) * kSlice;
    // the instruction reads 128 rows of A, past the end of a smaller stage: the last one keeps clear of the ring's end
    const uint32_t past = stage_bytes < kTileM * kSlice ? kTileM * kSlice - stage_bytes : 0;
    const int stages = min(kMaxStages, static_cast<int>((kRing - past) / stage_bytes));
    Work w;
    w.first = first;
    w.count = count;
    w.padded = padded;
    w.prefix = prefix;
    w.E = a.E;
    w.M = a.M;
    w.N = a.N;
    w.k_slices = (a.K + kElems - 1) / kElems;
    w.cols = P == kGated ? bn / 2 : bn;
    w.n_tiles = (a.N + w.cols - 1) / w.cols;
    w.tiles = m_tiles * w.n_tiles;
    __syncthreads();
    const uint32_t tmem = sh->tmem;
    const bool run = sh->stop == 0;

    if (run && warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; i < w.tiles && ok; i += gridDim.x) {
                const Tile t = locate<P>(w, i);
                const int live = P == kDw ? kTileM : min(kTileM, t.count - t.m0);
                const int pieces = live > 64 ? 0 : (live + 15) / 16;  // 0: one copy of 128 rows
                const uint32_t bytes = (pieces ? pieces * 16 : kTileM) * kSlice + bn * kSlice;
                for (int k = 0; k < t.slices; ++k) {
                    if (!(ok = wait(a, sh, &sh->empty[s], phase ^ 1u))) break;
                    uint8_t* sa = ring + s * stage_bytes;
                    uint8_t* sb = sa + a_bytes;
                    uint64_t* bar = &sh->full[s];
                    mbar_arrive_expect_tx(bar, bytes);
                    const int at = k * kElems;
                    if constexpr (P == kDw) {
                        const int row = static_cast<int>(t.first) + k * 64;
                        for (int j = 0; j < 2; ++j) tensor_load_2d(sa + j * 8192, &map_a, t.m0 + 64 * j, row, bar);
                        for (int j = 0; j < bn / 64; ++j)
                            tensor_load_2d(sb + j * 8192, &map_b, t.n0 + 64 * j, row, bar);
                    } else {
                        const int row = static_cast<int>(t.first) + t.m0;
                        if (pieces == 0) tensor_load_2d(sa, &map_a, at, row, bar);
                        for (int j = 0; j < pieces; ++j)
                            tensor_load_2d(sa + j * 16 * kSlice, &map_a16, at, row + 16 * j, bar);
                        if constexpr (P == kGated) {
                            for (int j = 0; j < bn / 64; ++j) {
                                tensor_load_3d(sb + j * 4096, &map_b, at, t.n0 + 32 * j, 2 * t.e, bar);
                                tensor_load_3d(sb + bn * (kSlice / 2) + j * 4096, &map_b, at, t.n0 + 32 * j,
                                               2 * t.e + 1, bar);
                            }
                        } else if constexpr (P == kDown) {
                            for (int j = 0; j < bn / 64; ++j)
                                tensor_load_3d(sb + j * 8192, &map_b, at, t.n0 + 64 * j, t.e, bar);
                        } else {
                            for (int j = 0; j < bn / 64; ++j)
                                tensor_load_3d(sb + j * 8192, &map_b, t.n0 + 64 * j, at, t.e, bar);
                        }
                    }
                    ++issued;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok)  // let the copies in flight land before the block's shared memory goes
                for (int64_t j = max(int64_t(0), issued - stages); j < issued; ++j)
                    mbar_wait_bounded(&sh->full[j % stages], static_cast<uint32_t>((j / stages) & 1),
                                      static_cast<uint64_t>(a.timeout_ns));
        }
    } else if (run && warp == 1) {
        const uint32_t desc = mma_desc(FP8 ? 0u : 1u, kAmn, kBmn, kTileM, bn);
        int s = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < w.tiles && ok; i += gridDim.x) {
            const Tile t = locate<P>(w, i);
            if (t.slices == 0) continue;
            if (!(ok = wait(a, sh, &sh->acc_empty[buf], acc_phase ^ 1u))) break;
            tc_fence_after();
            for (int k = 0; k < t.slices; ++k) {
                if (!(ok = wait(a, sh, &sh->full[s], phase))) break;
                tc_fence_after();
                uint8_t* sa = ring + s * stage_bytes;
                uint8_t* sb = sa + a_bytes;
                int steps = 4;
                if constexpr (P == kDw) {
                    const int valid = min(64, t.count - 64 * k);
                    steps = (valid + 15) / 16;
                    if (valid < steps * 16) {  // rows past the group: zero in both operands
                        const int boxes = 2 + bn / 64, chunks = (steps * 16 - valid) * 8;
                        for (int j = lane; j < boxes * chunks; j += 32) {
                            uint8_t* box = j / chunks < 2 ? sa + j / chunks * 8192 : sb + (j / chunks - 2) * 8192;
                            *reinterpret_cast<uint4*>(box + valid * kSlice + j % chunks * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    const uint64_t da = operand_desc(smem_addr(sa), kAmn ? 8192 : 16, 1024);
                    const uint64_t db = operand_desc(smem_addr(sb), kBmn ? 8192 : 16, 1024);
                    for (int j = 0; j < steps; ++j)  // 32 bytes of k, or 16 rows of it
                        mma<FP8>(tmem + buf * 256, da + j * ((kAmn ? 2048 : 32) >> 4),
                                 db + j * ((kBmn ? 2048 : 32) >> 4), desc, k > 0 || j > 0);
                    mma_commit(&sh->empty[s]);
                    if (k + 1 == t.slices) mma_commit(&sh->acc_full[buf]);
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if ((buf ^= 1) == 0) acc_phase ^= 1u;
        }
    } else if (run) {
        const int quarter = warp & 3;  // the rows of tensor memory a warp may read
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int64_t i = blockIdx.x; i < w.tiles; i += gridDim.x) {
            const Tile t = locate<P>(w, i);
            if (t.slices > 0) {
                if (!wait(a, sh, &sh->acc_full[buf], acc_phase)) break;
                tc_fence_after();
            }
            epilogue<P>(a, t, bn, tmem + buf * 256, quarter, lane, tid - 64);
            if (t.slices > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->acc_empty[buf]);
                if ((buf ^= 1) == 0) acc_phase ^= 1u;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_free(tmem, 512);
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

// One product: left operand's rows (and dw's right ones) or weights, as the kernel's maps want them.
template <int P, bool FP8 = false>
int launch_product(const void* left, const void* right, const moe::FfnArgs& a, cudaStream_t stream) {
    constexpr int bytes = FP8 ? 1 : 2;
    CUtensorMap map_a, map_a16, map_b;
    int rc;
    if constexpr (P == moe::kDw) {
        rc = moe_host::make_tensor_map(&map_a, left, 2, 2, a.M, a.rows, 1, 64);
        map_a16 = map_a;
        if (rc == MOE_OK) rc = moe_host::make_tensor_map(&map_b, right, 2, 2, a.N, a.rows, 1, 64);
    } else {
        rc = moe_host::make_tensor_map(&map_a, left, bytes, 2, a.K, a.rows, 1, moe::kTileM);
        if (rc == MOE_OK) rc = moe_host::make_tensor_map(&map_a16, left, bytes, 2, a.K, a.rows, 1, 16);
        if (rc == MOE_OK) {
            if constexpr (P == moe::kGated)
                rc = moe_host::make_tensor_map(&map_b, right, bytes, 3, a.K, a.N, 2 * a.E, 32);
            else if constexpr (P == moe::kDown)
                rc = moe_host::make_tensor_map(&map_b, right, 2, 3, a.K, a.N, a.E, 64);
            else
                rc = moe_host::make_tensor_map(&map_b, right, 2, 3, a.N, a.K, a.E, 64);
        }
    }
    if (rc != MOE_OK) return rc;
    const size_t smem = 1024 + moe::kRing + sizeof(moe::Shared) + sizeof(int) * (4 * static_cast<size_t>(a.E) + 1);
    static_assert(1024 + moe::kRing + sizeof(moe::Shared) + sizeof(int) * 4097 <= 227 * 1024, "shared memory");
    if (cudaFuncSetAttribute(moe::ffn_kernel<P, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    return moe_host::launch(moe::ffn_kernel<P, FP8>, dim3(static_cast<unsigned>(moe_host::num_sms())),
                            dim3(moe::kThreads), smem, stream, map_a, map_a16, map_b, a);
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
    a.timeout_ns = moe_host::timeout_ns();
    a.a_scale = x_scale;
    a.b_scale = w_scale;
    a.N = I;
    a.K = H;
    a.out = h;
    a.preact_out = preact;
    const int rg = fp8 ? launch_product<moe::kGated, true>(x, w_gate_up, a, stream)
                       : launch_product<moe::kGated>(x, w_gate_up, a, stream);
    if (rg != MOE_OK) return rg;
    a.a_scale = a.b_scale = nullptr;
    a.N = H;
    a.K = I;
    a.out = y;
    return launch_product<moe::kDown>(h, w_down, a, stream);
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
    a.timeout_ns = moe_host::timeout_ns();
    if (dx != nullptr || dw_gate_up != nullptr) {
        a.preact_in = preact;
        a.N = I;
        a.K = H;
        a.out = dgate_up;
        rc = launch_product<moe::kDgate>(dy, w_down, a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dx != nullptr) {
        a.N = H;
        a.K = 2 * I;
        a.out = dx;
        rc = launch_product<moe::kDx>(dgate_up, w_gate_up, a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dw_gate_up != nullptr) {
        a.M = 2 * I;
        a.N = H;
        a.out = dw_gate_up;
        rc = launch_product<moe::kDw>(dgate_up, x, a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dw_down != nullptr) {
        a.M = H;
        a.N = I;
        a.out = dw_down;
        rc = launch_product<moe::kDw>(dy, h, a, stream);
    }
    return rc;
}
