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
// One persistent kernel; two blocks on neighbouring SMs work as a pair on one
// tile (tcgen05 with cta_group::2, M = 256).  The instruction's M side is the
// weights' output index and its N side the group's rows: the weights' extents
// fill tiles of 256, while a group of any length is cut into tiles of equal
// length, a multiple of 16 rows up to 256, so that ragged groups cost little.
// (In dw both sides are weights' indexes and the groups are the k side.)
// Each block holds the fp32 accumulators of its 128 output channels by all the
// tile's rows in tensor memory, twice, so that one tile's epilogue runs under
// the next one's products.
//
// Warp 0 of each block brings its operands' slices of 128 bytes of k into a
// ring of shared-memory stages (tensor copies, 128-byte swizzle): 128 rows of
// the M side and half of the tile's N side, of which the hardware shows both
// halves to both SMs.  Warp 1 of the pair's first block issues the matrix
// instructions.  Warps 2-9 read the accumulators (a warp sees 32 channels),
// turn them through shared memory so that a row's channels lie side by side,
// and write the output.  In the gated product every 32 rows of the M side are
// 16 channels of the gate and the same 16 of the up projection, so that a
// warp has both for silu(g) * u; dgate applies the activation's gradient to
// dh there, so that dh is never written.
//
// Where k is the contiguous index (x, h, dy, dgate_up; weights of gated and
// down) a stage holds rows of 64 k's (128 in 8 bits); where it is not (weights
// of dgate and dx, both sides of dw) it holds rows of 64 of the M or N index,
// one for each k, and the instruction reads it transposed.  Slices that leave
// an array are filled with zeros by the copy.  In dw a group's last slice runs
// on into other rows, which may hold anything: a further warp of each block
// zeroes them in both operands.  It does so as soon as the slice is there,
// while the instructions of the slices before it run.
#include <cuda_fp8.h>

#include "tensor_core.cuh"
#include "vec8.cuh"

namespace moe {

enum Product { kGated, kDown, kDgate, kDx, kDw };

constexpr int kTile = 256;         // both sides of a tile at most
constexpr int kHalf = 128;         // a block's part of it
constexpr int kSlice = 128;        // bytes of a stage's row
constexpr int kMaxStages = 12;
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kMendWarp = 2 + kEpilogueWarps;  // dw has one warp more
constexpr int kChunk = 16;         // accumulator columns that a warp turns at a time
constexpr int kTurnStride = 48;    // floats between a chunk's rows: 16 banks apart for the gated reads

struct FfnArgs {
    const float* a_scale;   // gated in 8 bits: scales of x's rows and of the channels
    const float* b_scale;
    const float* preact_in;
    const int32_t* cu;
    const int32_t* count;
    int32_t* status;
    int64_t rows;
    int E, M, N, K;         // M: output channels; K: contraction length; dw: output M x N
    int ring_bytes;
    int wide;               // dw: rows of whole 32-byte sectors
    uint16_t* out;
    float* preact_out;
    int64_t timeout_ns;
};

struct Shared {
    float turn[kEpilogueWarps][kChunk * kTurnStride];
    uint64_t full[kMaxStages], empty[kMaxStages], tail_full[kMaxStages], tail_ready[kMaxStages], acc_full[2],
        acc_empty[2];
    uint32_t tmem;
    int stop;               // the plan's status held an error
    int scan[kMendWarp + 1], most[kMendWarp + 1];
};

struct Tile {
    int e;
    int first, count, padded;  // the group's first row, its rows, and with its padding
    int m0;                    // the pair's first output channel
    int n0, n;                 // first row within the group (dw: first column) and how many
    int slices;                // of k
    bool last;                 // the group's last rows
};

// What every warp of a block knows about the work.
struct Work {
    const int *first, *count, *padded;
    const int* prefix;  // row tiles before each expert (not dw)
    int E, M, N, k_slices;
    int m_step, m_tiles;
    int64_t tiles;
};

template <int P>
__device__ __forceinline__ Tile locate(const Work& w, int64_t t) {
    Tile r;
    int nt;
    int64_t at;
    if constexpr (P == kDw) {
        nt = (w.N + kTile - 1) / kTile;
        const int64_t per = static_cast<int64_t>(w.m_tiles) * nt;
        r.e = static_cast<int>(t / per);
        at = t - r.e * per;
    } else {
        int lo = 0, hi = w.E;  // the expert with prefix[e] * m_tiles <= t < prefix[e + 1] * m_tiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (static_cast<int64_t>(w.prefix[mid]) * w.m_tiles <= t) lo = mid;
            else hi = mid;
        }
        r.e = lo;
        nt = w.prefix[lo + 1] - w.prefix[lo];
        at = t - static_cast<int64_t>(w.prefix[lo]) * w.m_tiles;
    }
    // bands of 8 tiles of the N side, the M side outermost within a band: what
    // the pairs work on at one time is about square and stays in L2
    constexpr int kBand = 8;
    const int64_t per_band = static_cast<int64_t>(kBand) * w.m_tiles;
    const int band = static_cast<int>(at / per_band);
    const int in_band = static_cast<int>(at - band * per_band);
    const int width = min(kBand, nt - band * kBand);
    r.m0 = in_band / width * w.m_step;
    const int j = band * kBand + in_band % width;
    r.first = w.first[r.e];
    r.count = w.count[r.e];
    r.padded = w.padded[r.e];
    r.last = j == nt - 1;
    if constexpr (P == kDw) {
        r.n0 = j * kTile;
        r.n = min(kTile, w.N - r.n0);
        r.slices = (r.count + 63) / 64;
    } else {
        const int each = ((r.count + nt - 1) / nt + 15) & ~15;
        r.n0 = j * each;
        r.n = min(each, r.count - r.n0);
        r.slices = w.k_slices;
    }
    return r;
}

// Bounded wait; on a timeout the caller gives up and the plan's status says so.
__device__ __forceinline__ bool wait(const FfnArgs& a, uint64_t* bar, uint32_t parity) {
    if (mbar_wait_pair(bar, parity, static_cast<uint64_t>(a.timeout_ns))) return true;
    record_error(a.status, MOE_ERR_DEVICE_TIMEOUT, blockIdx.x);
    return false;
}

// silu(g) = g * sigmoid(g) and sigmoid(g).  The hardware exponential and
// division are within 2^-20 of the exact value for |g| < 16; beyond, where
// the sigmoid is 0 or 1 to bf16's precision or the result tiny, the relative
// error grows as |g| * 2^-24.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + __expf(-g)); }

__device__ __forceinline__ void store4_bf16(uint16_t* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(a, b), pack2(c, d));
}

// One chunk of a row product: 16 rows of the group by the warp's 32 channels,
// turned through `turn` so that neighbouring lanes hold neighbouring channels.
template <int P>
__device__ __forceinline__ void epilogue_chunk(const FfnArgs& a, const Tile& t, int rank, uint32_t acc, int c0,
                                               int quarter, int lane, float* turn) {
    const int64_t M = a.M;
    uint32_t v[kChunk];
    if constexpr (P == kGated) {
        const int c = t.m0 + rank * 64 + quarter * 16 + (lane & 3) * 4;  // this lane's 4 channels
        __syncwarp();
        tmem_load16(acc + c0, v);
        tmem_wait_load();
#pragma unroll
        for (int j = 0; j < kChunk; ++j) turn[j * kTurnStride + lane] = __uint_as_float(v[j]);
        __syncwarp();
#pragma unroll
        for (int it = 0; it < kChunk / 8; ++it) {
            const int j = it * 8 + (lane >> 2), n = c0 + j;
            if (n >= t.n || c >= M) continue;
            const int64_t row = t.first + static_cast<int64_t>(t.n0 + n);
            float4 g = *reinterpret_cast<const float4*>(turn + j * kTurnStride + (lane & 3) * 4);
            float4 u = *reinterpret_cast<const float4*>(turn + j * kTurnStride + 16 + (lane & 3) * 4);
            if (a.a_scale != nullptr) {
                const float s = __ldg(a.a_scale + row);
                const float4 sg = __ldg(reinterpret_cast<const float4*>(a.b_scale + 2 * M * t.e + c));
                const float4 su = __ldg(reinterpret_cast<const float4*>(a.b_scale + 2 * M * t.e + M + c));
                g = make_float4(g.x * (s * sg.x), g.y * (s * sg.y), g.z * (s * sg.z), g.w * (s * sg.w));
                u = make_float4(u.x * (s * su.x), u.y * (s * su.y), u.z * (s * su.z), u.w * (s * su.w));
            }
            if (a.preact_out != nullptr) {
                *reinterpret_cast<float4*>(a.preact_out + row * 2 * M + c) = g;
                *reinterpret_cast<float4*>(a.preact_out + row * 2 * M + M + c) = u;
            }
            store4_bf16(a.out + row * M + c, silu(g.x) * u.x, silu(g.y) * u.y, silu(g.z) * u.z, silu(g.w) * u.w);
        }
    } else {
        const int c = t.m0 + rank * kHalf + quarter * 32 + (lane & 7) * 4;
        constexpr int kIts = kChunk / 4;
        float4 g[P == kDgate ? kIts : 1], u[P == kDgate ? kIts : 1];
        if constexpr (P == kDgate) {  // asked for before the accumulators are read
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int n = c0 + it * 4 + (lane >> 3);
                if (n < t.n && c < M) {
                    const float* pre = a.preact_in + (t.first + static_cast<int64_t>(t.n0 + n)) * 2 * M + c;
                    g[it] = ld_stream_f4(pre);
                    u[it] = ld_stream_f4(pre + M);
                }
            }
        }
        __syncwarp();
        tmem_load16(acc + c0, v);
        tmem_wait_load();
#pragma unroll
        for (int j = 0; j < kChunk; ++j) turn[j * kTurnStride + lane] = __uint_as_float(v[j]);
        __syncwarp();
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
            const int j = it * 4 + (lane >> 3), n = c0 + j;
            if (n >= t.n || c >= M) continue;
            const int64_t row = t.first + static_cast<int64_t>(t.n0 + n);
            const float4 d = *reinterpret_cast<const float4*>(turn + j * kTurnStride + (lane & 7) * 4);
            if constexpr (P == kDgate) {
                const float dh[4] = {d.x, d.y, d.z, d.w}, gs[4] = {g[it].x, g[it].y, g[it].z, g[it].w},
                            us[4] = {u[it].x, u[it].y, u[it].z, u[it].w};
                float dg[4], du[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = sigmoid(gs[i]);
                    dg[i] = dh[i] * us[i] * s * fmaf(gs[i], 1.f - s, 1.f);
                    du[i] = dh[i] * gs[i] * s;
                }
                store4_bf16(a.out + row * 2 * M + c, dg[0], dg[1], dg[2], dg[3]);
                store4_bf16(a.out + row * 2 * M + M + c, du[0], du[1], du[2], du[3]);
            } else {
                store4_bf16(a.out + row * M + c, d.x, d.y, d.z, d.w);
            }
        }
    }
}

// dw: a lane holds an output row; it writes 16 columns of it.
__device__ __forceinline__ void epilogue_dw(const FfnArgs& a, const Tile& t, int rank, uint32_t acc, int c0, int quarter,
                                            int lane) {
    const int m = t.m0 + rank * kHalf + quarter * 32 + lane;
    uint32_t v[kChunk];
    if (t.slices > 0) {
        __syncwarp();
        tmem_load16(acc + c0, v);
        tmem_wait_load();
    } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] = 0u;
    }
    if (m >= a.M) return;
    uint16_t* out = a.out + (static_cast<int64_t>(t.e) * a.M + m) * a.N + t.n0 + c0;
    uint32_t p[kChunk / 2];
#pragma unroll
    for (int j = 0; j < kChunk; j += 2) p[j / 2] = pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
    if (a.wide) {  // whole 32-byte sectors
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out), "r"(p[0]), "r"(p[1]), "r"(p[2]),
                     "r"(p[3]), "r"(p[4]), "r"(p[5]), "r"(p[6]), "r"(p[7])
                     : "memory");
        return;
    }
    st_v4(out, make_uint4(p[0], p[1], p[2], p[3]));
    if (c0 + 8 < t.n) st_v4(out + 8, make_uint4(p[4], p[5], p[6], p[7]));
}

template <int P, bool FP8>
__global__ void __launch_bounds__(P == kDw ? kThreads + 32 : kThreads, 1)
    ffn_kernel(const __grid_constant__ CUtensorMap map_m, const __grid_constant__ CUtensorMap map_n,
               const __grid_constant__ CUtensorMap map_n16, const FfnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    constexpr bool kMmn = P == kDgate || P == kDx || P == kDw, kNmn = P == kDw;  // k is not the contiguous index
    constexpr int kElems = FP8 ? 128 : 64;                                       // k's of a slice

    uint8_t* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Shared* sh = reinterpret_cast<Shared*>(ring + a.ring_bytes);
    int* first = reinterpret_cast<int*>(sh + 1);
    int *count = first + a.E, *padded = count + a.E, *prefix = padded + a.E;  // prefix: E + 1

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(pair_rank());
    if (tid == 0) {
        tensor_prefetch(&map_m);
        tensor_prefetch(&map_n);
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
            mbar_init(&sh->tail_full[i], 1);
            mbar_init(&sh->tail_ready[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], 2 * kEpilogueWarps);
        }
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == 1) tmem_alloc(&sh->tmem, 512);
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh->stop = ld_volatile_s32(a.status) != 0;

    // ---- the groups: row tiles before each expert, and the longest group
    const int threads = P == kDw ? kThreads + 32 : kThreads, warps = threads / 32;
    const int per = (a.E + threads - 1) / threads;
    int mine = 0, longest = 0;
    for (int e = tid * per; e < min(a.E, (tid + 1) * per); ++e) {
        const int64_t f = __ldg(a.cu + e), c = __ldg(a.count + e), p = c == 0 ? 0 : __ldg(a.cu + e + 1) - f;
        const bool fits = c >= 0 && f >= 0 && p >= c && f + p <= a.rows;
        if (!fits) record_error(a.status, MOE_ERR_DEVICE_INDEX, e);
        first[e] = fits ? static_cast<int>(f) : 0;
        count[e] = fits ? static_cast<int>(c) : 0;
        padded[e] = fits ? static_cast<int>(p) : 0;
        mine += (count[e] + kTile - 1) / kTile;
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
    __syncthreads();
    int row_tiles = 0;
    before -= mine;
    longest = 0;
    for (int i = 0; i < warps; ++i) {
        if (i < warp) before += sh->scan[i];
        row_tiles += sh->scan[i];
        longest = max(longest, sh->most[i]);
    }
    for (int e = tid * per; e < min(a.E, (tid + 1) * per); ++e) {
        prefix[e] = before;
        before += (count[e] + kTile - 1) / kTile;
    }
    if (tid == 0) prefix[a.E] = row_tiles;

    Work w;
    w.first = first;
    w.count = count;
    w.padded = padded;
    w.prefix = prefix;
    w.E = a.E;
    w.M = a.M;
    w.N = a.N;
    w.k_slices = (a.K + kElems - 1) / kElems;
    w.m_step = P == kGated ? kHalf : kTile;  // a gated tile holds each channel twice
    w.m_tiles = (a.M + w.m_step - 1) / w.m_step;
    w.tiles = P == kDw ? static_cast<int64_t>(a.E) * w.m_tiles * ((a.N + kTile - 1) / kTile)
                       : static_cast<int64_t>(row_tiles) * w.m_tiles;
    // short groups leave room for more stages: the N side's part is as long as the longest tile's half
    const int half = (min(P == kDw ? kTile : longest, kTile) + 15) / 16 * 8;
    const int n_rows = P == kDw || half > 64 ? kHalf : max(16, (half + 15) / 16 * 16);
    const uint32_t stage_bytes = static_cast<uint32_t>(kHalf + n_rows) * kSlice;
    const int stages = min(kMaxStages, static_cast<int>(a.ring_bytes / stage_bytes));
    tc_fence_before();
    __syncthreads();
    pair_sync();  // both blocks' barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const bool run = sh->stop == 0;
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (run && warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t i = pair; i < w.tiles && ok; i += pairs) {
                const Tile t = locate<P>(w, i);
                const int mine = ((t.n + 15) & ~15) / 2;              // N-side rows (dw: columns) of a block
                const int pieces = P == kDw ? (mine + 63) / 64 : mine > 64 ? 0 : (mine + 15) / 16;
                const uint32_t bytes =
                    kHalf * kSlice + (P == kDw ? pieces * 8192 : pieces ? pieces * 16 * kSlice : kHalf * kSlice);
                const int m = t.m0 + rank * (P == kGated ? 64 : kHalf);
                for (int k = 0; k < t.slices; ++k) {
                    if (!(ok = wait(a, &sh->empty[s], phase ^ 1u))) break;
                    uint8_t* sm = ring + s * stage_bytes;
                    uint8_t* sn = sm + kHalf * kSlice;
                    // both blocks' copies are counted by the first one's barrier, but those
                    // of a slice that has to be mended by each block's own
                    uint32_t bar;
                    if (P == kDw && k + 1 == t.slices && (t.count & 15) != 0) {
                        mbar_arrive_expect_tx(&sh->tail_full[s], bytes);
                        bar = smem_addr(&sh->tail_full[s]);
                    } else if (rank == 0) {
                        mbar_arrive_expect_tx(&sh->full[s], 2 * bytes);
                        bar = smem_addr(&sh->full[s]);
                    } else {
                        bar = leader_addr(&sh->full[s]);
                    }
                    const int at = k * kElems;
                    if constexpr (P == kGated) {
                        for (int j = 0; j < 4; ++j) tensor_load_4d(sm + j * 4096, &map_m, at, m + 16 * j, 0, t.e, bar);
                    } else if constexpr (P == kDown) {
                        tensor_load_3d(sm, &map_m, at, m, t.e, bar);
                    } else if constexpr (P == kDw) {
                        for (int j = 0; j < 2; ++j)
                            tensor_load_2d(sm + j * 8192, &map_m, m + 64 * j, t.first + k * 64, bar);
                    } else {
                        for (int j = 0; j < 2; ++j) tensor_load_3d(sm + j * 8192, &map_m, m + 64 * j, at, t.e, bar);
                    }
                    if constexpr (P == kDw) {
                        for (int j = 0; j < pieces; ++j)
                            tensor_load_2d(sn + j * 8192, &map_n, t.n0 + rank * mine + 64 * j, t.first + k * 64, bar);
                    } else {
                        const int row = t.first + t.n0 + rank * mine;
                        if (pieces == 0) tensor_load_2d(sn, &map_n, at, row, bar);
                        for (int j = 0; j < pieces; ++j)
                            tensor_load_2d(sn + j * 16 * kSlice, &map_n16, at, row + 16 * j, bar);
                    }
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {  // time for the copies in flight to land before the block's shared memory goes
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 20000000u) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (run && warp == 1 && rank == 0) {
        // One thread from end to end, the four instructions of a slice unrolled:
        // gaps between them cost (a loop over a slice's steps: dw 1650 us, this 1430
        // at 32768 rows, H = I = 4096, 8 experts).
        if (lane == 0) {
            int s = 0, buf = 0;
            uint32_t acc_phase = 0, full_phase = 0, tail_phase = 0;  // the latter two: a bit a stage
            bool ok = true;
            for (int64_t i = pair; i < w.tiles && ok; i += pairs) {
                const Tile t = locate<P>(w, i);
                if (t.slices == 0) continue;
                const uint32_t desc = mma_desc(FP8 ? 0u : 1u, kMmn, kNmn, kTile, (t.n + 15) & ~15);
                const uint32_t acc = tmem + buf * kTile;
                if (!(ok = wait(a, &sh->acc_empty[buf], acc_phase ^ 1u))) break;
                for (int k = 0; k < t.slices; ++k) {
                    const bool last = k + 1 == t.slices;
                    if (P == kDw && last && (t.count & 15) != 0) {
                        if (!(ok = wait(a, &sh->tail_ready[s], (tail_phase >> s) & 1u))) break;
                        tail_phase ^= 1u << s;
                    } else {
                        if (!(ok = wait(a, &sh->full[s], (full_phase >> s) & 1u))) break;
                        full_phase ^= 1u << s;
                    }
                    tc_fence_after();
                    const uint32_t sm = smem_addr(ring + s * stage_bytes);
                    const uint64_t dm = operand_desc(sm, kMmn ? 8192 : 16, 1024);
                    const uint64_t dn = operand_desc(sm + kHalf * kSlice, kNmn ? 8192 : 16, 1024);
                    constexpr int kStepM = (kMmn ? 2048 : 32) >> 4, kStepN = (kNmn ? 2048 : 32) >> 4;
                    // 32 bytes of k, or 16 rows of it, an instruction; dw's last slice may have fewer
                    const int steps = P == kDw && last ? ((t.count - 1) % 64) / 16 + 1 : 4;
                    if (P != kDw || steps == 4) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma<FP8>(acc, dm + j * kStepM, dn + j * kStepN, desc, k > 0 || j > 0);
                    } else {
                        for (int j = 0; j < steps; ++j)
                            mma<FP8>(acc, dm + j * kStepM, dn + j * kStepN, desc, k > 0 || j > 0);
                    }
                    mma_commit(&sh->empty[s]);
                    if (last) mma_commit(&sh->acc_full[buf]);
                    if (++s == stages) s = 0;
                }
                if ((buf ^= 1) == 0) acc_phase ^= 1u;
            }
        }
        __syncwarp();
    } else if (P == kDw && run && warp == kMendWarp) {
        int s = 0;
        uint32_t tail_phase = 0;
        for (int64_t i = pair; i < w.tiles; i += pairs) {
            const Tile t = locate<P>(w, i);
            if (t.slices == 0) continue;
            s = (s + t.slices - 1) % stages;
            if ((t.count & 15) != 0) {
                if (!wait(a, &sh->tail_full[s], (tail_phase >> s) & 1u)) break;
                tail_phase ^= 1u << s;
                // rows from the group's end to a multiple of 16; the N side's boxes of
                // 64 columns follow the M side's two in the stage
                const int valid = t.count & 63, chunks = (((valid + 15) & ~15) - valid) * 8;
                const int boxes = 2 + (((t.n + 15) & ~15) / 2 + 63) / 64;
                uint8_t* at = ring + s * stage_bytes + valid * kSlice;
                for (int j = lane; j < boxes * chunks; j += 32)
                    *reinterpret_cast<uint4*>(at + j / chunks * 8192 + j % chunks * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(&sh->tail_ready[s]);
            }
            if (++s == stages) s = 0;
        }
    } else if (run && warp >= 2 && warp < kMendWarp) {
        const int quarter = warp & 3;           // the lanes of tensor memory that a warp may read
        const int turn = (warp - 2) >> 2;       // two warps a quarter take every other chunk
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int64_t i = pair; i < w.tiles; i += pairs) {
            const Tile t = locate<P>(w, i);
            if (t.slices > 0) {
                if (!wait(a, &sh->acc_full[buf], acc_phase)) break;
                tc_fence_after();
            }
            for (int c = turn * kChunk; c < t.n; c += 2 * kChunk) {
                if constexpr (P == kDw) epilogue_dw(a, t, rank, tmem + buf * kTile + lanes, c, quarter, lane);
                else epilogue_chunk<P>(a, t, rank, tmem + buf * kTile + lanes, c, quarter, lane, sh->turn[warp - 2]);
            }
            if (t.slices > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(&sh->acc_empty[buf]);
                if ((buf ^= 1) == 0) acc_phase ^= 1u;
            }
            if constexpr (P == kDown || P == kDx) {  // the group's padding: zeros
                if (t.last && t.padded > t.count) {
                    const int c0 = t.m0 + rank * kHalf, chunks = (min(kHalf, a.M - c0) + 7) / 8;
                    const int64_t todo = chunks > 0 ? static_cast<int64_t>(t.padded - t.count) * chunks : 0;
                    for (int64_t j = tid - 64; j < todo; j += 32 * kEpilogueWarps)
                        st_v4(a.out + (t.first + t.count + j / chunks) * static_cast<int64_t>(a.M) + c0 + 8 * (j % chunks),
                              make_uint4(0u, 0u, 0u, 0u));
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    pair_sync();  // neither block leaves while the other may still use its barriers or tensor memory
    if (warp == 1) {
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

// One product: the weights (dw: the left rows) and the rows (dw: the right ones).
template <int P, bool FP8 = false>
int launch_product(const void* weights, const void* row_data, moe::FfnArgs a, cudaStream_t stream) {
    constexpr int bytes = FP8 ? 1 : 2;
    CUtensorMap map_m, map_n, map_n16;
    int rc;
    if constexpr (P == moe::kGated) rc = moe_host::make_tensor_map(&map_m, weights, bytes, {a.K, a.M, 2, a.E}, 16, 2);
    else if constexpr (P == moe::kDown) rc = moe_host::make_tensor_map(&map_m, weights, 2, {a.K, a.M, a.E}, moe::kHalf);
    else if constexpr (P == moe::kDw) rc = moe_host::make_tensor_map(&map_m, weights, 2, {a.M, a.rows}, 64);
    else rc = moe_host::make_tensor_map(&map_m, weights, 2, {a.M, a.K, a.E}, 64);
    if (rc == MOE_OK)
        rc = P == moe::kDw ? moe_host::make_tensor_map(&map_n, row_data, 2, {a.N, a.rows}, 64)
                           : moe_host::make_tensor_map(&map_n, row_data, bytes, {a.K, a.rows}, moe::kHalf);
    if (rc == MOE_OK && P != moe::kDw) rc = moe_host::make_tensor_map(&map_n16, row_data, bytes, {a.K, a.rows}, 16);
    if (rc != MOE_OK) return rc;
    if (P == moe::kDw) map_n16 = map_n;
    // six stages of 32 KB with up to 256 experts, five beyond (their table takes the room)
    constexpr size_t kSmem = 227 * 1024, kStage = 2 * moe::kHalf * moe::kSlice;
    const size_t fixed = 1024 + sizeof(moe::Shared) + sizeof(int) * (4 * static_cast<size_t>(a.E) + 1);
    a.ring_bytes = static_cast<int>((kSmem - fixed) / kStage * kStage);
    a.wide = a.N % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    static_assert(1024 + sizeof(moe::Shared) + sizeof(int) * 4097 + 5 * kStage <= kSmem, "shared memory");
    if (cudaFuncSetAttribute(moe::ffn_kernel<P, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem)) != cudaSuccess)
        return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(moe_host::num_sms() & ~1));
    cfg.blockDim = dim3(P == moe::kDw ? moe::kThreads + 32 : moe::kThreads);
    cfg.dynamicSmemBytes = fixed + a.ring_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = moe_host::pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, moe::ffn_kernel<P, FP8>, map_m, map_n, map_n16, a) == cudaSuccess ? MOE_OK
                                                                                                    : MOE_ERR_CUDA;
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
    a.M = I;
    a.K = H;
    a.out = h;
    a.preact_out = preact;
    const int rg = fp8 ? launch_product<moe::kGated, true>(w_gate_up, x, a, stream)
                       : launch_product<moe::kGated>(w_gate_up, x, a, stream);
    if (rg != MOE_OK) return rg;
    a.a_scale = a.b_scale = nullptr;
    a.M = H;
    a.K = I;
    a.out = y;
    return launch_product<moe::kDown>(w_down, h, a, stream);
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
        a.M = I;
        a.K = H;
        a.out = dgate_up;
        rc = launch_product<moe::kDgate>(w_down, dy, a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dx != nullptr) {
        a.M = H;
        a.K = 2 * I;
        a.out = dx;
        rc = launch_product<moe::kDx>(w_gate_up, dgate_up, a, stream);
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
