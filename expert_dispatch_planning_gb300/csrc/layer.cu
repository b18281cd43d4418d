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
    int* sums;                   // [warps] of the scan
    float* weight;               // [N*K]
    uint16_t* place;             // [E] a chosen expert's place
    uint8_t* token;              // [N*K]
    int count;

    static __host__ __device__ int slots(int N, int K, int E) { return N * K < E ? N * K : E; }
    static __host__ __device__ size_t bytes(int N, int K, int E) {
        const size_t s = 8 * static_cast<size_t>(E) + 4 * (2 * slots(N, K, E) + 1) + 4 * kLayerWarps + 4 * N * K + 2 * E + N * K;
        return (s + 15) / 16 * 16;
    }
    __device__ Chosen(uint8_t* smem, const LayerArgs& a) {
        const int n = slots(a.N, a.K, a.E);
        tokens = reinterpret_cast<unsigned long long*>(smem);
        expert = reinterpret_cast<int*>(tokens + a.E);
        begin = expert + n;
        sums = begin + n + 1;
        weight = reinterpret_cast<float*>(sums + kLayerWarps);
        place = reinterpret_cast<uint16_t*>(weight + a.N * a.K);
        token = reinterpret_cast<uint8_t*>(place + a.E);
    }
    __device__ int size(int i) const { return begin[i + 1] - begin[i]; }

    // Reads topk_idx and topk_w once; `clear` comes before.
    __device__ void clear(const LayerArgs& a) {
        for (int e = threadIdx.x; e < a.E; e += kLayerThreads) tokens[e] = 0;
        __syncthreads();
    }
    __device__ void find(const LayerArgs& a) {
        constexpr int kMost = MOE_LAYER_MAX_TOKENS * 32 / kLayerThreads;  // pairs a thread
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pairs = a.N * a.K;
        int e_of[kMost];
        float w_of[kMost];
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int f = tid + i * kLayerThreads;
            e_of[i] = -1;
            if (f < pairs) {
                e_of[i] = a.topk_idx[f];
                w_of[i] = a.topk_w[f];
            }
        }
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (static_cast<unsigned>(e_of[i]) < static_cast<unsigned>(a.E))
                atomicOr(&tokens[e_of[i]], 1ull << ((tid + i * kLayerThreads) / a.K));
        __syncthreads();
        // a thread has a run of experts: chosen ones and pairs before it, in one word
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
        int i = before >> 16, at = before & 0xffff;
        for (int e = e0; e < e0 + per && e < a.E; ++e) {
            if (tokens[e] == 0) continue;
            expert[i] = e;
            begin[i] = at;
            place[e] = static_cast<uint16_t>(i);
            ++i;
            at += __popcll(tokens[e]);
        }
        if (tid == 0) begin[count] = all & 0xffff;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kMost; ++v)
            if (static_cast<unsigned>(e_of[v]) < static_cast<unsigned>(a.E)) {
                const int s = (tid + v * kLayerThreads) / a.K;
                const int p = begin[place[e_of[v]]] + __popcll(tokens[e_of[v]] & ((1ull << s) - 1));
                token[p] = static_cast<uint8_t>(s);
                weight[p] = w_of[v];
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
// A warp's ring of weight steps in shared memory, filled by its own copies (cp.async): no
// other warp waits for it, and it runs on over the ends of tiles and experts, so that memory
// is kept busy while the warps join their sums.  A step is kStepBytes of each of the warp's MT
// sixteens of rows.  Eight lanes copy a row's 128 bytes, a whole line (with the four lanes a
// row that a fragment has, 64 bytes of eight rows, memory gave a third less).
constexpr int kStepBytes = 128;
constexpr int kPieces = 2;  // of 64 bytes: what a fragment has of a row

// Rows of one tile: MT times two eights; eight h of sixteen m begins at first + m * tile + h * half.
struct WeightRows {
    const uint8_t* first;
    int64_t row, half, tile;  // bytes from one to the next
    int n;                    // rows that are there: of each half (gate and up), or of all
};

template <int MT, bool HALVES, int DEPTH>  // HALVES: n counts the rows of each half
struct WeightRing {
    static constexpr int kStep = MT * 16 * kStepBytes;
    static constexpr int kDepth = DEPTH;
    static constexpr int kWarpBytes = DEPTH * kStep;
    const uint32_t mine;
    int slot = 0;  // the step's that is read next
    __device__ explicit WeightRing(const uint8_t* smem) : mine(smem_addr(smem) + (threadIdx.x >> 5) * kWarpBytes) {}
    // 16-byte chunk `chunk` of row `row` of eight `e`: odd rows are turned by half a row, so that
    // the eight lanes of a read, two rows' four chunks, are in different banks.
    static __device__ __forceinline__ int place(int e, int row, int chunk) {
        return (e * 8 + row) * kStepBytes + (chunk ^ (row & 1) << 2) * 16;
    }
    // The step at byte `at` of the rows; zeros behind a row's end (`bytes`) and for rows that are not there.
    __device__ __forceinline__ void fetch(int ahead, const WeightRows& w, int at, int bytes) const {
        const int s = slot + ahead, r = (threadIdx.x & 31) >> 3, chunk = threadIdx.x & 7, k = at + chunk * 16;
        const uint32_t to = mine + (s >= DEPTH ? s - DEPTH : s) * kStep;
        __syncwarp();  // all lanes have read what was there
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = 4 * i + r;
                    const bool in = (HALVES ? 8 * m : 16 * m + 8 * half) + row < w.n && k < bytes;
                    const uint8_t* from = w.first + m * w.tile + half * w.half + row * w.row + k;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + place(2 * m + half, row, chunk)),
                                 "l"(in ? from : w.first), "r"(in ? 16 : 0)
                                 : "memory");
                }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        __syncwarp();
    }
    // The lane's piece p of its row (g) of an eight.
    __device__ __forceinline__ uint4 read(int m, int half, int p) const {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(mine + slot * kStep + place(2 * m + half, g, 4 * p + t))
                     : "memory");
        return v;
    }
    __device__ __forceinline__ void next() { slot = slot + 1 == DEPTH ? 0 : slot + 1; }
};

constexpr int kEights = 2;             // of tokens that a pass over a tile's weights takes
constexpr int kPass = 8 * kEights;

// The lane's token rows for the steps of a pass: both pieces of its token in each eight, asked
// for a step ahead.  A row that is not there is null and gives zeros.
struct Tokens {
    const uint8_t* row[kEights];
    uint4 v[kPieces][kEights];
    bool more;  // a second eight
    __device__ __forceinline__ void rows(const Chosen& c, int expert, int pass, const uint8_t* base, bool by_place,
                                         int64_t bytes) {
        const int first = c.begin[expert] + pass * kPass, cols = c.begin[expert + 1] - first;
        more = cols > 8;
#pragma unroll
        for (int j = 0; j < kEights; ++j) {
            const int p = 8 * j + ((threadIdx.x & 31) >> 2);
            row[j] = nullptr;
            if (p < cols) row[j] = base + (by_place ? first + p : c.token[first + p]) * bytes + (threadIdx.x & 3) * 16;
        }
    }
    __device__ __forceinline__ void load(int step, int bytes) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int at = step * kStepBytes + 64 * p;
            const bool in = at + static_cast<int>(threadIdx.x & 3) * 16 < bytes;
            v[p][0] = load16(row[0] + at, in && row[0] != nullptr);
            if (more) v[p][1] = load16(row[1] + at, in && row[1] != nullptr);
        }
    }
};

// One step: acc += the step's weight rows times tokens.
template <bool Q, int MT, typename Ring>
__device__ __forceinline__ void multiply(float (&acc)[MT][kEights][4], const Ring& ring, const uint4 (&v)[kPieces][kEights],
                                         bool more) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const Fragment<Q> b0(v[p][0]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const Fragment<Q> lo(ring.read(m, 0, p)), hi(ring.read(m, 1, p));
            product<Q>(acc[m][0], lo, hi, b0);
            if (more) product<Q>(acc[m][1], lo, hi, Fragment<Q>(v[p][1]));
        }
    }
}

template <int MT>
__device__ __forceinline__ void zero(float (&acc)[MT][kEights][4]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < kEights; ++j) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.f;
}

// ---------------------------------------------------------------- gate and up
__device__ __forceinline__ float silu(float g) {
    const float e = expf(-fabsf(g));
    return g * __fdiv_rn(g >= 0.f ? 1.f : e, 1.f + e);
}

constexpr int kGateUpTiles = 2;  // eights of channels in a tile
constexpr int kGateUpChannels = 8 * kGateUpTiles;
using GateUpRing = WeightRing<kGateUpTiles, true, 3>;

// A walk over a block's run of the chosen experts' channels: tile by tile (channels of one
// expert), pass by pass (sixteen of its tokens; the passes after the first find the tile's
// weights in L2), and over the warp's steps of k.
struct GateUpWalk {
    int64_t at, end;
    int expert, channel, n;  // the tile at hand: its place among the chosen, first channel, channels
    int pass, passes, step;
    __device__ void tile(const Chosen& c, int I) {
        pass = 0;
        passes = 0;
        if (at >= end) return;
        expert = static_cast<int>(at / I);
        channel = static_cast<int>(at - static_cast<int64_t>(expert) * I);
        n = I - channel < kGateUpChannels ? I - channel : kGateUpChannels;
        if (end - at < n) n = static_cast<int>(end - at);
        passes = (c.size(expert) + kPass - 1) / kPass;
    }
    // To the next pass or tile; whether there is one.
    __device__ bool next(const Chosen& c, int I) {
        if (++pass < passes) return true;
        at += n;
        tile(c, I);
        return at < end;
    }
};

// The warp's steps are kLayerWarps apart: what the block's warps ask for at one time is contiguous.
template <bool Q>
struct GateUpWeights {
    GateUpWalk walk;
    WeightRows w;
    __device__ void rows(const LayerArgs& a, const Chosen& c) {
        if (walk.at >= walk.end) return;
        w.row = static_cast<int64_t>(a.H) * (Q ? 1 : 2);
        w.half = a.I * w.row;
        w.tile = 8 * w.row;
        w.n = walk.n;
        w.first = static_cast<const uint8_t*>(a.w_gate_up) +
                  (static_cast<int64_t>(c.expert[walk.expert]) * 2 * a.I + walk.channel) * w.row;
    }
    __device__ __forceinline__ void fetch(const LayerArgs& a, const Chosen& c, const GateUpRing& ring, int ahead, int warp,
                                          int steps) {
        if (walk.at < walk.end && warp < steps) {
            ring.fetch(ahead, w, walk.step * kStepBytes, a.H * (Q ? 1 : 2));
            if ((walk.step += kLayerWarps) >= steps) {
                walk.step = warp;
                walk.next(c, a.I);
                rows(a, c);
            }
        }
        GateUpRing::commit();
    }
};

// The parts of a tile's pass are joined over the block's warps in `sum` ([warps][kGateUpTiles][32]),
// one eight of tokens after the other; warp m joins eight m of the channels.
template <bool Q>
__device__ __forceinline__ void gate_up_join(const LayerArgs& a, const Chosen& c, float4* sum, const GateUpWalk& walk,
                                             const float (&acc)[kGateUpTiles][kEights][4]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int e = c.expert[walk.expert], first = c.begin[walk.expert] + walk.pass * kPass,
              cols = c.begin[walk.expert + 1] - first;
#pragma unroll
    for (int j = 0; j < kEights; ++j) {
        if (8 * j >= cols) break;
        __syncthreads();  // the sums before are taken
#pragma unroll
        for (int m = 0; m < kGateUpTiles; ++m)
            sum[(warp * kGateUpTiles + m) * 32 + lane] = make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
        __syncthreads();
        if (warp >= kGateUpTiles) continue;
        float4 s = sum[warp * 32 + lane];
#pragma unroll
        for (int k = 1; k < kLayerWarps; ++k) {
            const float4 o = sum[(k * kGateUpTiles + warp) * 32 + lane];
            s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
        }
        const int row = 8 * warp + g, ch = walk.channel + row;
        if (row >= walk.n) continue;
        float wg = 1.f, wu = 1.f;
        if constexpr (Q) {
            wg = __ldg(a.w_scale + static_cast<int64_t>(e) * 2 * a.I + ch);
            wu = __ldg(a.w_scale + static_cast<int64_t>(e) * 2 * a.I + a.I + ch);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int p = 8 * j + 2 * t + v;
            if (p >= cols) continue;
            float gate = v == 0 ? s.x : s.y, up = v == 0 ? s.z : s.w;
            if constexpr (Q) {
                const float xs = __ldg(a.x_scale + c.token[first + p]);
                gate = gate * wg * xs;
                up = up * wu * xs;
            }
            const __nv_bfloat16 h = __float2bfloat16_rn(silu(gate) * up);
            a.h[static_cast<int64_t>(first + p) * a.I + ch] = __bfloat16_as_ushort(h);
        }
    }
}

template <bool Q>
__global__ void __launch_bounds__(kLayerThreads, 2) layer_gate_up_kernel(const LayerArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    GateUpRing ring(smem);
    float4* sum = reinterpret_cast<float4*>(smem + kLayerWarps * GateUpRing::kWarpBytes);
    Chosen c(reinterpret_cast<uint8_t*>(sum + kLayerWarps * kGateUpTiles * 32), a);
    c.clear(a);
    pdl_wait();
    pdl_trigger();
    c.find(a);
    const int warp = threadIdx.x >> 5, bytes = a.H * (Q ? 1 : 2), steps = (bytes + kStepBytes - 1) / kStepBytes;
    const uint8_t* x = static_cast<const uint8_t*>(a.x);
    // every block takes an equal run of the chosen experts' channels
    const int64_t all = static_cast<int64_t>(c.count) * a.I;
    GateUpWalk walk;
    walk.at = blockIdx.x * all / gridDim.x;
    walk.end = (blockIdx.x + 1) * all / gridDim.x;
    walk.step = warp;
    walk.tile(c, a.I);
    if (walk.at >= walk.end) return;
    GateUpWeights<Q> weights;
    weights.walk = walk;
    weights.rows(a, c);
    for (int i = 0; i < GateUpRing::kDepth - 1; ++i) weights.fetch(a, c, ring, i, warp, steps);
    GateUpWalk ahead = walk;  // the tokens', a step ahead
    Tokens tokens;
    tokens.rows(c, walk.expert, 0, x, false, bytes);
    if (warp < steps) tokens.load(warp, bytes);
    do {
        float acc[kGateUpTiles][kEights][4];
        zero(acc);
        for (int s = warp; s < steps; s += kLayerWarps) {
            weights.fetch(a, c, ring, GateUpRing::kDepth - 1, warp, steps);
            uint4 now[kPieces][kEights];
            const bool more = tokens.more;
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
#pragma unroll
                for (int j = 0; j < kEights; ++j) now[p][j] = tokens.v[p][j];
            if (s + kLayerWarps < steps) {
                tokens.load(s + kLayerWarps, bytes);
            } else if (ahead.next(c, a.I)) {
                tokens.rows(c, ahead.expert, ahead.pass, x, false, bytes);
                tokens.load(warp, bytes);
            }
            GateUpRing::wait();
            multiply<Q>(acc, ring, now, more);
            ring.next();
        }
        gate_up_join<Q>(a, c, sum, walk, acc);
    } while (walk.next(c, a.I));
}

// ---------------------------------------------------------------- down
// A walk over a warp's run of the chosen experts' steps of k: one expert's (its part) after the
// other, pass by pass.
struct DownWalk {
    int at, end, steps;
    int expert, first, last;  // the part at hand: the expert's place among the chosen, its steps
    int pass, passes, step;
    __device__ void part(const Chosen& c) {
        pass = 0;
        passes = 0;
        if (at >= end) return;
        expert = at / steps;
        step = first = at - expert * steps;
        last = end - at < steps - first ? first + end - at : steps;
        passes = (c.size(expert) + kPass - 1) / kPass;
    }
    __device__ bool next(const Chosen& c) {
        step = first;
        if (++pass < passes) return true;
        at += last - first;
        part(c);
        return at < end;
    }
};

// Sixteens of rows that a cluster has.  The sums of more than eight tokens leave room for one.
template <bool MANY>
struct Down {
    static constexpr int kTiles = MANY ? 1 : 2;
    static constexpr int kRows = 16 * kTiles;
    using Ring = WeightRing<kTiles, false, MANY ? 4 : 3>;
};

template <bool MANY>
struct DownWeights {
    using D = Down<MANY>;
    DownWalk walk;
    WeightRows w;
    int first_row;
    __device__ void rows(const LayerArgs& a, const Chosen& c) {
        if (walk.at >= walk.end) return;
        w.row = static_cast<int64_t>(a.I) * 2;
        w.half = 8 * w.row;
        w.tile = 16 * w.row;
        w.n = a.H - first_row;
        w.first = reinterpret_cast<const uint8_t*>(a.w_down) +
                  (static_cast<int64_t>(c.expert[walk.expert]) * a.H + first_row) * w.row;
    }
    __device__ __forceinline__ void fetch(const LayerArgs& a, const Chosen& c, const typename D::Ring& ring, int ahead) {
        if (walk.at < walk.end) {
            ring.fetch(ahead, w, walk.step * kStepBytes, 2 * a.I);
            if (++walk.step >= walk.last) {
                walk.next(c);
                rows(a, c);
            }
        }
        D::Ring::commit();
    }
};

// A part's products, weighted, are added to the warp's sums [rows][N].
template <int MT>
__device__ __forceinline__ void down_add(const LayerArgs& a, const Chosen& c, float* sum, const DownWalk& walk,
                                         const float (&acc)[MT][kEights][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int first = c.begin[walk.expert] + walk.pass * kPass, cols = c.begin[walk.expert + 1] - first;
#pragma unroll
    for (int j = 0; j < kEights; ++j)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int p = 8 * j + 2 * t + v;
            if (p >= cols) continue;
            const float w = c.weight[first + p];
            float* s = sum + c.token[first + p];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float* o = s + (16 * m + 8 * half + g) * a.N;
                    *o = fmaf(w, acc[m][j][2 * half + v], *o);
                }
        }
    __syncwarp();  // the next expert's tokens are other lanes'
}

__device__ __forceinline__ float load_cluster(const float* p, uint32_t rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// A cluster has Down::kRows rows of the output; all warps of its blocks share the chosen experts' k.
template <bool MANY>
__global__ void __launch_bounds__(kLayerThreads, 2) layer_down_kernel(const LayerArgs a) {
    using D = Down<MANY>;
    extern __shared__ __align__(16) uint8_t smem[];
    typename D::Ring ring(smem);
    float* sums = reinterpret_cast<float*>(smem + kLayerWarps * D::Ring::kWarpBytes);  // [warps][rows][N]
    Chosen c(reinterpret_cast<uint8_t*>(sums) + sizeof(float) * kLayerWarps * D::kRows * a.N, a);
    const int tid = threadIdx.x, warp = tid >> 5;
    uint32_t rank, blocks;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(blocks));
    for (int v = tid; v < kLayerWarps * D::kRows * a.N; v += kLayerThreads) sums[v] = 0.f;
    // topk_idx and the weights come from before the launch that this one may overlap
    c.clear(a);
    c.find(a);
    const uint8_t* h = reinterpret_cast<const uint8_t*>(a.h);
    const int bytes = 2 * a.I;
    DownWalk walk;
    walk.steps = (bytes + kStepBytes - 1) / kStepBytes;
    const int64_t all = static_cast<int64_t>(c.count) * walk.steps, me = rank * kLayerWarps + warp, of = blocks * kLayerWarps;
    walk.at = static_cast<int>(me * all / of);
    walk.end = static_cast<int>((me + 1) * all / of);
    walk.part(c);
    DownWeights<MANY> weights;
    weights.walk = walk;
    weights.first_row = blockIdx.x / blocks * D::kRows;
    weights.rows(a, c);
    for (int i = 0; i < D::Ring::kDepth - 1; ++i) weights.fetch(a, c, ring, i);
    pdl_wait();
    pdl_trigger();
    if (walk.at < walk.end) {
        float* sum = sums + warp * D::kRows * a.N;
        DownWalk ahead = walk;  // the tokens', a step ahead
        Tokens tokens;
        tokens.rows(c, walk.expert, 0, h, true, bytes);
        tokens.load(walk.first, bytes);
        do {
            float acc[D::kTiles][kEights][4];
            zero(acc);
            for (int s = walk.first; s < walk.last; ++s) {
                weights.fetch(a, c, ring, D::Ring::kDepth - 1);
                uint4 now[kPieces][kEights];
                const bool more = tokens.more;
#pragma unroll
                for (int p = 0; p < kPieces; ++p)
#pragma unroll
                    for (int j = 0; j < kEights; ++j) now[p][j] = tokens.v[p][j];
                if (s + 1 < walk.last) {
                    tokens.load(s + 1, bytes);
                } else if (ahead.next(c)) {
                    tokens.rows(c, ahead.expert, ahead.pass, h, true, bytes);
                    tokens.load(ahead.first, bytes);
                }
                D::Ring::wait();
                multiply<false>(acc, ring, now, more);
                ring.next();
            }
            down_add(a, c, sum, walk, acc);
        } while (walk.next(c));
    }
    __syncthreads();
    for (int v = tid; v < D::kRows * a.N; v += kLayerThreads) {
        float o = sums[v];
#pragma unroll
        for (int w = 1; w < kLayerWarps; ++w) o += sums[w * D::kRows * a.N + v];
        sums[v] = o;
    }
    // the blocks' sums are joined in their order, each block an equal part of them
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int v = rank * kLayerThreads + tid; v < D::kRows * a.N; v += blocks * kLayerThreads) {
        const int row = v % D::kRows, s = v / D::kRows;  // neighbouring threads write neighbouring elements
        if (weights.first_row + row >= a.H) continue;
        float o = 0.f;
        for (uint32_t r = 0; r < blocks; ++r) o += load_cluster(sums + row * a.N + s, r);
        a.out[static_cast<int64_t>(s) * a.H + weights.first_row + row] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
    }
    // a block's sums stay until the others have read them
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace moe

// ---------------------------------------------------------------- host
namespace {

using namespace moe_host;
using moe::LayerArgs;

template <bool Q>
int launch_gate_up(const LayerArgs& a, cudaStream_t stream) {
    const size_t smem = moe::kLayerWarps * (moe::GateUpRing::kWarpBytes + sizeof(float4) * moe::kGateUpTiles * 32) +
                        moe::Chosen::bytes(a.N, a.K, a.E);
    if (cudaFuncSetAttribute(moe::layer_gate_up_kernel<Q>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    return launch(moe::layer_gate_up_kernel<Q>, dim3(static_cast<unsigned>(2 * num_sms())), dim3(moe::kLayerThreads),
                  smem, stream, a);
}

template <bool MANY>
int launch_down(const LayerArgs& a, cudaStream_t stream) {
    using D = moe::Down<MANY>;
    const size_t smem = moe::kLayerWarps * (D::Ring::kWarpBytes + sizeof(float) * D::kRows * a.N) +
                        moe::Chosen::bytes(a.N, a.K, a.E);
    if (cudaFuncSetAttribute(moe::layer_down_kernel<MANY>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    const int groups = (a.H + D::kRows - 1) / D::kRows;
    int blocks = 1;  // of a cluster: as many as keep all resident
    while (blocks < 8 && 2 * blocks * groups <= 2 * num_sms()) blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(groups * blocks));
    cfg.blockDim = dim3(moe::kLayerThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, moe::layer_down_kernel<MANY>, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
    const int up = q ? launch_gate_up<true>(a, stream) : launch_gate_up<false>(a, stream);
    if (up != MOE_OK) return up;
    return N > 8 ? launch_down<true>(a, stream) : launch_down<false>(a, stream);
}
