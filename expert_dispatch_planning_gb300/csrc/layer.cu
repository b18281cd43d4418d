// layer.cu -- a whole mixture-of-experts layer for a few tokens (sm_103a).
//
// For N <= 64 tokens: the router's choice, and for every chosen pair (s, k)
// with e = idx[s][k]
//   g = x[s] . w_gate[e]^T,  u = x[s] . w_up[e]^T,  h = bf16(silu(g) * u),
//   out[s] = bf16(sum over k of w[s][k] * (h . w_down[e]^T)).
// A decoding step reads the weights of every chosen expert for a handful of
// rows: memory bounds it.  So nothing is permuted or padded; the weights stream
// from memory once, through rings in shared memory that each warp fills and
// reads by itself, and everything else hides behind them.
//
// Measured (GB300, copy rate 6.80 TB/s; from run to run): 61 tokens, 64 experts of
// 4096 x 1280, 321 to 328 us, 6.1 to 6.3 TB/s; three tokens, 24 experts of 7168 x 1024
// in 8 bits, 109 to 115 us, 6.0 to 6.3 TB/s.  One token, 8 experts of 2048 x 768: 23 us
// of which the weights take 11; the rest is the launches' starts and ends, one after the
// other.  Narrow experts are further off: k is dealt to a block's warps anew for each
// tile, so that with fewer than eight steps of 128 bytes some load nothing (17 tokens, 60
// experts of 1000 x 712: 1.6 times the weights' time; 64 tokens, 64 of 2048 x 96: 4.3).
//
// Launches: the router's, gate/up, down; for more than eight tokens the down product's
// parts are summed by a fourth.  Each block finds the chosen experts and their tokens by
// itself from topk_idx (a 64-bit set of tokens for every expert).
//
// Products.  mma.m16n8k16 with 16 weight rows as its M side and up to 8 tokens
// as its N side: an expert has a few tokens, and a tcgen05 tile of 64 or 128
// rows would leave most SMs without one.  A lane's place in the fragment wants
// 2 + 2 elements of a row for every 16 of k; since a sum may be taken in any
// order of k, as long as both operands agree, a lane takes 16 contiguous bytes
// of its row and of its token's instead, with no shuffles.  A tile is 32 rows, so that
// a token's bytes serve four times the weights' (16 rows: 61 tokens 495 us against
// 370).  8-bit operands become fp16 in registers (exact), their products are exact in the
// fp32 accumulator.
#include <cmath>

#include "vec8.cuh"

namespace moe {

constexpr int kLayerThreads = 256;
constexpr int kLayerWarps = kLayerThreads / 32;
// At most, in layer_down_kernel, whose sums are [warps][rows][N].  (By tiles of rows and a sum, as for more tokens, the
// layer takes 29.3 us for one token and 95 for eight, of 128 experts of 2048 x 768; so 23.7 and 85.5.)
constexpr int kDownTokens = 8;

struct LayerArgs {
    const void* x;
    const float* x_scale;
    const void* w_gate_up;
    const float* w_scale;
    const uint16_t* w_down;
    const int32_t* topk_idx;
    const float* topk_w;
    uint16_t* h;  // [N*K][I], rows in the order of experts, then tokens
    float* y;     // [N*K][H], for many tokens
    uint16_t* out;
    int N, K, E, H, I;
};

// Code.  While weights stream through L2 they push the kernels' own instructions out of it,
// and then every 128 bytes of code that run for the first time cost some 45 ns, on all SMs at
// once.  So what runs before the first weights are asked for is short: loops are not unrolled,
// and steps that happen in two places are one place in the code (61 tokens, 64 experts of
// 4096 x 1280: 354 us before, 330 so; the router within these blocks: one token 38 us, 28 in its
// shortest form, against 24 with its own launch).

// ---------------------------------------------------------------- the chosen experts
// In shared memory: expert[i] and begin[i] of the i-th chosen expert (begin[count] = pairs),
// and for every place its pair, token and weight.
struct Chosen {
    unsigned long long* tokens;  // [E] sets of tokens
    int* expert;                 // [slots]
    int* begin;                  // [slots + 1]
    int* sums;                   // [warps] of the scan
    float* weight;               // [N*K]
    uint16_t* place;             // [E] a chosen expert's place
    uint16_t* pair;              // [N*K] flat indices s * K + k
    uint8_t* token;              // [N*K]

    static __host__ __device__ int slots(int N, int K, int E) { return N * K < E ? N * K : E; }
    static __host__ __device__ size_t bytes(int N, int K, int E) {
        const size_t s = 8 * static_cast<size_t>(E) + 4 * (2 * slots(N, K, E) + 1) + 4 * kLayerWarps + 7 * N * K + 2 * E;
        return (s + 15) / 16 * 16;
    }
    __device__ Chosen(uint8_t* smem, int N, int K, int E) {
        const int n = slots(N, K, E);
        tokens = reinterpret_cast<unsigned long long*>(smem);
        expert = reinterpret_cast<int*>(tokens + E);
        begin = expert + n;
        sums = begin + n + 1;
        weight = reinterpret_cast<float*>(sums + kLayerWarps);
        place = reinterpret_cast<uint16_t*>(weight + N * K);
        pair = place + E;
        token = reinterpret_cast<uint8_t*>(pair + N * K);
    }
    __device__ int size(int i) const { return begin[i + 1] - begin[i]; }
};

// Fills `smem` as Chosen's arrays from the router's outputs; returns the number of chosen experts.
// All threads call.
__device__ __noinline__ int choose(uint8_t* smem, int N, int K, int E, const int32_t* topk_idx, const float* topk_w) {
    const Chosen c(smem, N, K, E);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pairs = N * K;
    // Up to 32 pairs: one warp, a lane a pair, experts in the order of their first pairs (one token, 8 of 128 experts
    // of 2048 x 768: 23.5 us, 24.8 without; four tokens 52.5 and 54.4).
    if (pairs <= 32) {
        if (warp == 0) {
            int e = -1 - lane;  // of no pair: unlike any other
            float w = 0.f;
            if (lane < pairs) {
                const int i = topk_idx[lane];
                w = topk_w[lane];
                if (static_cast<unsigned>(i) < static_cast<unsigned>(E)) e = i;
            }
            const unsigned same = __match_any_sync(FULL_MASK, e), below = (1u << lane) - 1;
            const int leader = __ffs(same) - 1;
            const bool leads = e >= 0 && leader == lane;
            const unsigned leaders = __ballot_sync(FULL_MASK, leads);
            int before = leads ? __popc(same) : 0;  // pairs of this leader and those ahead of it
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(FULL_MASK, before, o);
                if (lane >= o) before += t;
            }
            const int all = __shfl_sync(FULL_MASK, before, 31);
            const int first = __shfl_sync(FULL_MASK, before, leader) - __popc(same);
            if (leads) {
                const int i = __popc(leaders & below);
                c.expert[i] = e;
                c.begin[i] = first;
            }
            if (e >= 0) {
                const int p = first + __popc(same & below);
                c.token[p] = static_cast<uint8_t>(lane / K);
                c.pair[p] = static_cast<uint16_t>(lane);
                c.weight[p] = w;
            }
            if (lane == 0) {
                c.begin[__popc(leaders)] = all;
                c.sums[0] = __popc(leaders);
            }
        }
        __syncthreads();
        return c.sums[0];
    }
#pragma unroll 1
    for (int e = tid; e < E; e += kLayerThreads) c.tokens[e] = 0;
    __syncthreads();
    auto chosen = [&](int f) {  // the pair's expert; -1 for an index that the router does not give
        const int e = topk_idx[f];
        return static_cast<unsigned>(e) < static_cast<unsigned>(E) ? e : -1;
    };
#pragma unroll 1
    for (int f = tid; f < pairs; f += kLayerThreads) {
        const int e = chosen(f);
        if (e >= 0) atomicOr(&c.tokens[e], 1ull << (f / K));
    }
    __syncthreads();
    // a thread has a run of experts: chosen ones and pairs before it, in one word
    const int per = (E + kLayerThreads - 1) / kLayerThreads, e0 = tid * per, e1 = e0 + per < E ? e0 + per : E;
    int mine = 0;
#pragma unroll 1
    for (int e = e0; e < e1; ++e)
        if (c.tokens[e] != 0) mine += 0x10000 + __popcll(c.tokens[e]);
    int before = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(FULL_MASK, before, o);
        if (lane >= o) before += t;
    }
    if (lane == 31) c.sums[warp] = before;
    __syncthreads();
    int all = 0;
    before -= mine;
#pragma unroll 1
    for (int w = 0; w < kLayerWarps; ++w) {
        if (w < warp) before += c.sums[w];
        all += c.sums[w];
    }
    const int count = all >> 16;
    int i = before >> 16, at = before & 0xffff;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
        if (c.tokens[e] == 0) continue;
        c.expert[i] = e;
        c.begin[i] = at;
        c.place[e] = static_cast<uint16_t>(i);
        ++i;
        at += __popcll(c.tokens[e]);
    }
    if (tid == 0) c.begin[count] = all & 0xffff;
    __syncthreads();
#pragma unroll 1
    for (int f = tid; f < pairs; f += kLayerThreads) {
        const int e = chosen(f);
        if (e < 0) continue;
        const int s = f / K, p = c.begin[c.place[e]] + __popcll(c.tokens[e] & ((1ull << s) - 1));
        c.token[p] = static_cast<uint8_t>(s);
        c.pair[p] = static_cast<uint16_t>(f);
        c.weight[p] = topk_w[f];
    }
    __syncthreads();
    return count;
}

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
            if constexpr (Q)
                asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                    : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
                    : "r"(u[i]));
            else
                w[i] = u[i];
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
    for (int i = 0; i < (Q ? 8 : 4); i += 2) mma<Q>(c, lo.w[i], hi.w[i], lo.w[i + 1], hi.w[i + 1], b.w[i], b.w[i + 1]);
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

// Rows of one tile: MT times two eights of them.
struct WeightRows {
    const uint8_t* any;        // an address to give where nothing is read
    const uint8_t* lane;       // chunk lane % 8 of row lane / 8 of the first eight
    int64_t four, half, tile;  // bytes from a row to its fourth next, an eight to the other, a sixteen to the next
    int n;                     // rows that are there: of each half (gate and up), or of all
    __device__ __forceinline__ void set(const void* base, int64_t first_row, int64_t row, int there) {
        n = there;
        any = static_cast<const uint8_t*>(base);
        lane = any + (first_row + ((threadIdx.x & 31) >> 3)) * row + (threadIdx.x & 7) * 16;
    }
};

template <int MT, bool HALVES, int DEPTH>  // HALVES: n counts the rows of each half
struct WeightRing {
    static constexpr int kStep = MT * 16 * kStepBytes;
    static constexpr int kDepth = DEPTH;
    static constexpr int kWarpBytes = DEPTH * kStep;
    // A row's 16-byte chunks lie one after the other, an odd row's turned by half a row: so the
    // eight lanes of a read, two rows' four chunks, are in different banks.
    uint32_t to;       // where the lane's copies go: row r = lane / 8 of each four rows, chunk lane % 8
    uint32_t from;     // where its pieces are: row g = lane / 4 of each eight, chunk lane % 4 (the other piece: ^ 64)
    uint32_t at = 0;   // the step's that is read next, and the one that is filled next
    uint32_t fill = 0;
    __device__ explicit WeightRing(const uint8_t* smem) {
        const uint32_t lane = threadIdx.x & 31, mine = smem_addr(smem) + (threadIdx.x >> 5) * kWarpBytes;
        const uint32_t r = lane >> 3, chunk = lane & 7, g = lane >> 2, t = lane & 3;
        to = mine + r * kStepBytes + (chunk ^ (r & 1) << 2) * 16;
        from = mine + g * kStepBytes + (t ^ (g & 1) << 2) * 16;
    }
    // The step at byte `k` of the rows; zeros behind a row's end (`bytes`) and for rows that are not there.
    // What is not read `again` is the first to leave L2, before tokens, h and the kernels' code
    // (61 tokens, 64 experts of 4096 x 1280: 327 us, 338 without; the 8-bit case of the header 108 to 113, 117 to 121).
    __device__ __forceinline__ void fetch(const WeightRows& w, int k, int bytes, bool again) {
        const int r = (threadIdx.x & 31) >> 3, mine = k + static_cast<int>(threadIdx.x & 7) * 16;
        const uint8_t* first = w.lane + k;
        uint64_t once, kept;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(kept));
        const uint64_t policy = again ? kept : once;
        const uint32_t slot = to + fill;
        fill = fill == (DEPTH - 1) * kStep ? 0 : fill + kStep;
        __syncwarp();  // all lanes have read what was there
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint8_t* eight = first + m * w.tile + half * w.half;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool in = (HALVES ? 8 * m : 16 * m + 8 * half) + 4 * i + r < w.n && mine < bytes;
                    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2, %3;" ::"r"(
                                     slot + (4 * (2 * m + half) + 2 * i) * 256),
                                 "l"(in ? eight + i * w.four : w.any), "r"(in ? 16 : 0), "l"(policy)
                                 : "memory");
                }
            }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        __syncwarp();
    }
    // The lane's piece p of its row of an eight.
    __device__ __forceinline__ uint4 read(int m, int half, int p) const {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"((from ^ p << 6) + at + (2 * m + half) * 1024)
                     : "memory");
        return v;
    }
    __device__ __forceinline__ void next() { at = at == (DEPTH - 1) * kStep ? 0 : at + kStep; }
};

// The lane's token rows for the steps of a pass over a tile's weights, which takes up to EIGHTS eights
// of an expert's tokens: both pieces of its token in each eight, asked for a step ahead.  A row that is
// not there is null and gives zeros.
template <int EIGHTS>
struct Tokens {
    const uint8_t* row[EIGHTS];
    uint4 v[kPieces][EIGHTS];
    bool more;  // than one eight
    __device__ __forceinline__ void rows(const Chosen& c, int expert, int pass, const uint8_t* base, bool by_place,
                                         int64_t bytes) {
        const int first = c.begin[expert] + pass * 8 * EIGHTS, cols = c.begin[expert + 1] - first;
        more = cols > 8;
#pragma unroll
        for (int j = 0; j < EIGHTS; ++j) {
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
#pragma unroll
            for (int j = 0; j < EIGHTS; ++j)
                if (j == 0 || more) v[p][j] = load16(row[j] + at, in && row[j] != nullptr);
        }
    }
};

// One step: acc += the step's weight rows times tokens.
template <bool Q, int MT, int EIGHTS, typename Ring>
__device__ __forceinline__ void multiply(float (&acc)[MT][EIGHTS][4], const Ring& ring, const uint4 (&v)[kPieces][EIGHTS],
                                         bool more) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const Fragment<Q> b0(v[p][0]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const Fragment<Q> lo(ring.read(m, 0, p)), hi(ring.read(m, 1, p));
            product<Q>(acc[m][0], lo, hi, b0);
            if constexpr (EIGHTS > 1)
                if (more) product<Q>(acc[m][1], lo, hi, Fragment<Q>(v[p][1]));
        }
    }
}

template <int MT, int EIGHTS>
__device__ __forceinline__ void zero(float (&acc)[MT][EIGHTS][4]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < EIGHTS; ++j) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.f;
}

__device__ __forceinline__ float silu(float g) {
    const float e = expf(-fabsf(g));
    return g * __fdiv_rn(g >= 0.f ? 1.f : e, 1.f + e);
}

// ---------------------------------------------------------------- rows by rows
// Gate and up, and the down product of many tokens: every block takes an equal run of the chosen
// experts' rows (channels of gate and up: a row of each), its warps share k.
constexpr int kTiles = 2;  // sixteens of rows in a tile
template <bool DOWN>
using TileRing = WeightRing<kTiles, !DOWN, 3>;

// A walk over a block's run: tile by tile (32 rows of one expert, or 16 channels with two rows
// each), pass by pass (those after the first find the tile's weights in L2), and over the warp's
// steps of k, which are kLayerWarps apart: what the block's warps ask for at one time is contiguous.
template <bool DOWN, int EIGHTS>
struct TileWalk {
    static constexpr int kUnits = DOWN ? 16 * kTiles : 8 * kTiles;
    int left;             // units (rows or channels) of the run from this tile on; 0: the walk has ended
    int expert, unit, n;  // the tile at hand: its expert's place among the chosen, first unit, their number
    int pass, passes, step;
    bool fresh;           // nothing has been derived from the tile or pass yet
    __device__ __forceinline__ void tile(const Chosen& c, int units) {
        n = units - unit < kUnits ? units - unit : kUnits;
        if (left < n) n = left;
        pass = 0;
        passes = (c.size(expert) + 8 * EIGHTS - 1) / (8 * EIGHTS);
    }
    // To the next pass or tile; whether there is one.
    __device__ __forceinline__ bool next(const Chosen& c, int units) {
        fresh = true;
        if (++pass < passes) return true;
        left -= n;
        if (left == 0) return false;
        unit += n;
        if (unit == units) {
            unit = 0;
            ++expert;
        }
        tile(c, units);
        return true;
    }
    // To the warp's next step.
    __device__ __forceinline__ void advance(const Chosen& c, int units, int warp, int steps) {
        if ((step += kLayerWarps) < steps) return;
        step = warp;
        next(c, units);
    }
};

// The parts of a tile's pass are joined over the block's warps in `sum` ([warps][kTiles][32]), one
// eight of tokens after the other; warp m joins sixteen m of the rows.  A lane has two tokens of rows
// g and g + 8, which for gate and up are the two rows of a channel.
template <bool Q, bool DOWN, int EIGHTS>
__device__ __forceinline__ void join(const LayerArgs& a, const Chosen& c, float4* sum, const TileWalk<DOWN, EIGHTS>& walk,
                                     const float (&acc)[kTiles][EIGHTS][4]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int e = c.expert[walk.expert], first = c.begin[walk.expert] + walk.pass * 8 * EIGHTS,
              cols = c.begin[walk.expert + 1] - first;
#pragma unroll
    for (int j = 0; j < EIGHTS; ++j) {
        if (8 * j >= cols) break;
        __syncthreads();  // the sums before are taken
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
            sum[(warp * kTiles + m) * 32 + lane] = make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
        __syncthreads();
        if (warp >= kTiles) continue;
        float4 s = sum[warp * 32 + lane];
#pragma unroll
        for (int k = 1; k < kLayerWarps; ++k) {
            const float4 o = sum[(k * kTiles + warp) * 32 + lane];
            s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
        }
        if constexpr (DOWN) {
            const int row = 16 * warp + g;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int p = 8 * j + 2 * t + v;
                if (p >= cols) continue;
                const float w = c.weight[first + p];
                float* y = a.y + static_cast<int64_t>(c.pair[first + p]) * a.H + walk.unit;
                if (row < walk.n) y[row] = w * (v == 0 ? s.x : s.y);
                if (row + 8 < walk.n) y[row + 8] = w * (v == 0 ? s.z : s.w);
            }
        } else {
            const int row = 8 * warp + g, ch = walk.unit + row;
            if (row >= walk.n) continue;
            float wg = 1.f, wu = 1.f;
            if constexpr (Q) {
                wg = ld_stream_f32(a.w_scale + static_cast<int64_t>(e) * 2 * a.I + ch);
                wu = ld_stream_f32(a.w_scale + static_cast<int64_t>(e) * 2 * a.I + a.I + ch);
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int p = 8 * j + 2 * t + v;
                if (p >= cols) continue;
                float gate = v == 0 ? s.x : s.y, up = v == 0 ? s.z : s.w;
                if constexpr (Q) {
                    const float xs = ld_stream_f32(a.x_scale + c.token[first + p]);
                    gate = gate * wg * xs;
                    up = up * wu * xs;
                }
                // rounded once: the down product's operand, of w_down's type, as in moe_expert_ffn (out is 0.0023 from
                // 64 bits, 0.0017 if h were not rounded; as two bf16 it would take twice the products and bytes of h)
                const __nv_bfloat16 h = __float2bfloat16_rn(silu(gate) * up);
                a.h[static_cast<int64_t>(first + p) * a.I + ch] = __bfloat16_as_ushort(h);
            }
        }
    }
}

// DOWN: y[s*K + k] = w[s][k] * (h . w_down^T) in fp32.  Else h.  EIGHTS: of tokens, in a pass.
template <bool Q, bool DOWN, int EIGHTS>
__global__ void __launch_bounds__(kLayerThreads, 2) layer_rows_kernel(const LayerArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    using Ring = TileRing<DOWN>;
    Ring ring(smem);
    float4* sum = reinterpret_cast<float4*>(smem + kLayerWarps * Ring::kWarpBytes);
    uint8_t* lists = reinterpret_cast<uint8_t*>(sum + kLayerWarps * kTiles * 32);
    const Chosen c(lists, a.N, a.K, a.E);
    if constexpr (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    // (of the down product topk_idx and the weights come from before the launch that this one may overlap)
    const int count = choose(lists, a.N, a.K, a.E, a.topk_idx, a.topk_w);
    const int warp = threadIdx.x >> 5, units = DOWN ? a.H : a.I;
    const int bytes = DOWN ? 2 * a.I : a.H * (Q ? 1 : 2), steps = (bytes + kStepBytes - 1) / kStepBytes;
    const uint8_t* x = static_cast<const uint8_t*>(DOWN ? a.h : a.x);
    const unsigned all = static_cast<unsigned>(count) * units, per = all / gridDim.x, rest = all - per * gridDim.x;
    const unsigned begin = blockIdx.x * per + (blockIdx.x < rest ? blockIdx.x : rest);
    TileWalk<DOWN, EIGHTS> walk;
    walk.left = static_cast<int>(per + (blockIdx.x < rest ? 1 : 0));
    if (DOWN && (walk.left == 0 || warp >= steps)) {
        pdl_wait();
        pdl_trigger();
    }
    if (walk.left == 0) return;
    walk.expert = static_cast<int>(begin / units);
    walk.unit = static_cast<int>(begin) - walk.expert * units;
    walk.step = warp;
    walk.fresh = true;
    walk.tile(c, units);
    TileWalk<DOWN, EIGHTS> weights = walk, ahead = walk;  // the ring's, and the tokens', a step ahead
    WeightRows w;
    Tokens<EIGHTS> tokens;
    float acc[kTiles][EIGHTS][4];
    zero(acc);
    int lead = warp < steps ? Ring::kDepth - 1 : 0;  // steps to ask for before the first product
    while (true) {
        if (warp < steps) {
            if (weights.left != 0) {
                if (weights.fresh) {
                    const int64_t row = DOWN ? 2 * static_cast<int64_t>(a.I) : static_cast<int64_t>(a.H) * (Q ? 1 : 2);
                    w.four = 4 * row;
                    w.half = DOWN ? 8 * row : a.I * row;
                    w.tile = DOWN ? 16 * row : 8 * row;
                    const int64_t first = static_cast<int64_t>(c.expert[weights.expert]) * (DOWN ? a.H : 2 * a.I) + weights.unit;
                    w.set(DOWN ? static_cast<const void*>(a.w_down) : a.w_gate_up, first, row, weights.n);
                    weights.fresh = false;
                }
                ring.fetch(w, weights.step * kStepBytes, bytes, weights.pass + 1 < weights.passes);
                weights.advance(c, units, warp, steps);
            }
            Ring::commit();
            if (lead > 1) {
                --lead;
                continue;
            }
            if (DOWN && lead == 1) {
                pdl_wait();
                pdl_trigger();
            }
            uint4 now[kPieces][EIGHTS];
            const bool more = tokens.more;
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
#pragma unroll
                for (int j = 0; j < EIGHTS; ++j) now[p][j] = tokens.v[p][j];
            if (ahead.left != 0) {
                if (ahead.fresh) {
                    tokens.rows(c, ahead.expert, ahead.pass, x, DOWN, bytes);
                    ahead.fresh = false;
                }
                tokens.load(ahead.step, bytes);
                ahead.advance(c, units, warp, steps);
            }
            if (lead == 1) {
                lead = 0;
                continue;
            }
            Ring::wait();
            multiply<Q>(acc, ring, now, more);
            ring.next();
        }
        if ((walk.step += kLayerWarps) >= steps) {
            join<Q, DOWN>(a, c, sum, walk, acc);
            if (!walk.next(c, units)) break;
            zero(acc);
            walk.step = warp;
        }
    }
}

// out[s] = bf16 of the sum of its pairs' y, in the order of k: a thread eight elements.
__global__ void __launch_bounds__(256) layer_sum_kernel(const LayerArgs a) {
    pdl_wait();
    pdl_trigger();
    const int nvec = a.H / 8;
    const int v = blockIdx.x * 256 + threadIdx.x;
    if (v >= a.N * nvec) return;
    const int s = v / nvec, c = v - s * nvec;
    const float4* y = reinterpret_cast<const float4*>(a.y + static_cast<int64_t>(s) * a.K * a.H) + 2 * c;
    float f[8] = {};
#pragma unroll 4
    for (int k = 0; k < a.K; ++k) {
        const float4 p = y[static_cast<int64_t>(k) * (a.H / 4)], q = y[static_cast<int64_t>(k) * (a.H / 4) + 1];
        f[0] += p.x, f[1] += p.y, f[2] += p.z, f[3] += p.w;
        f[4] += q.x, f[5] += q.y, f[6] += q.z, f[7] += q.w;
    }
    store8(a.out + static_cast<int64_t>(s) * a.H, c, f);
}

// ---------------------------------------------------------------- down, few tokens
// A walk over a warp's run of the chosen experts' steps of k: one expert's (its part) after the other.
struct DownWalk {
    int left, steps;   // steps of the run from this one on; an expert's
    int expert, step;  // the expert's place among the chosen, the step of it
    bool fresh;        // nothing has been derived from the expert yet
    // To the next step; whether it begins another expert or the run has ended.
    __device__ __forceinline__ bool advance() {
        if (++step == steps) {
            step = 0;
            ++expert;
            fresh = true;
        }
        return --left == 0 || step == 0;
    }
};

constexpr int kDownRows = 16 * kTiles, kDownBlocks = 4;  // of a cluster: rows, and blocks at most
using DownRing = WeightRing<kTiles, false, 3>;

// A part's products, weighted, are added to the warp's sums [rows][N].
__device__ __forceinline__ void down_add(const LayerArgs& a, const Chosen& c, float* sum, int expert,
                                         const float (&acc)[kTiles][1][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int first = c.begin[expert], cols = c.size(expert);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int p = 2 * t + v;
        if (p >= cols) continue;
        const float w = c.weight[first + p];
        float* s = sum + c.token[first + p];
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float* o = s + (16 * m + 8 * half + g) * a.N;
                *o = fmaf(w, acc[m][0][2 * half + v], *o);
            }
    }
    __syncwarp();  // the next expert's tokens are other lanes'
}

// Into the memory of the cluster's first block.
__device__ __forceinline__ void store_first(float* p, float v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_addr(p)));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// A cluster has `rows` rows of the output, at most kDownRows; all warps of its blocks share the
// chosen experts' k.  (Where a token's sum is cut so depends on how many experts all tokens chose: its
// last bits may change with the others.  layer_rows_kernel's do not.)
__global__ void __launch_bounds__(kLayerThreads, 2) layer_down_kernel(const LayerArgs a, int rows) {
    extern __shared__ __align__(128) uint8_t smem[];
    DownRing ring(smem);
    float* sums = reinterpret_cast<float*>(smem + kLayerWarps * DownRing::kWarpBytes);  // [warps][rows][N]
    float* parts = sums + kLayerWarps * kDownRows * a.N;  // [blocks of a cluster][rows][N], of the first
    uint8_t* lists = reinterpret_cast<uint8_t*>(parts + kDownBlocks * kDownRows * a.N);
    const Chosen c(lists, a.N, a.K, a.E);
    const int tid = threadIdx.x, warp = tid >> 5;
    uint32_t rank, blocks;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(blocks));
    // (waited for before the first write into another block's memory, which has to run by then)
    if (blocks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
#pragma unroll 1
    for (int v = tid; v < kLayerWarps * kDownRows * a.N; v += kLayerThreads) sums[v] = 0.f;
    // topk_idx and the weights come from before the launch that this one may overlap
    const int count = choose(lists, a.N, a.K, a.E, a.topk_idx, a.topk_w);
    const uint8_t* h = reinterpret_cast<const uint8_t*>(a.h);
    const int bytes = 2 * a.I, first_row = static_cast<int>(blockIdx.x / blocks) * rows;
    const int there = a.H - first_row < rows ? a.H - first_row : rows;
    // equal parts of the steps, to a step, for the cluster's warps
    DownWalk walk;
    walk.steps = (bytes + kStepBytes - 1) / kStepBytes;
    const unsigned all = static_cast<unsigned>(count) * walk.steps, me = rank * kLayerWarps + warp, of = blocks * kLayerWarps;
    const unsigned per = all / of, rest = all - per * of, begin = me * per + (me < rest ? me : rest);
    walk.left = static_cast<int>(per + (me < rest ? 1 : 0));
    walk.expert = static_cast<int>(begin / walk.steps);
    walk.step = static_cast<int>(begin) - walk.expert * walk.steps;
    walk.fresh = true;
    DownWalk weights = walk, ahead = walk;  // the ring's, and the tokens', a step ahead
    WeightRows w;
    Tokens<1> tokens;
    float* sum = sums + warp * kDownRows * a.N;
    float acc[kTiles][1][4];
    zero(acc);
    int lead = DownRing::kDepth - 1;  // steps to ask for before the first product
    while (walk.left != 0 || lead != 0) {
        if (weights.left != 0) {
            if (weights.fresh) {
                const int64_t row = bytes;
                w.four = 4 * row;
                w.half = 8 * row;
                w.tile = 16 * row;
                w.set(a.w_down, static_cast<int64_t>(c.expert[weights.expert]) * a.H + first_row, row, there);
                weights.fresh = false;
            }
            ring.fetch(w, weights.step * kStepBytes, bytes, false);
            weights.advance();
        }
        DownRing::commit();
        if (lead > 1) {
            --lead;
            continue;
        }
        if (lead == 1) {
            pdl_wait();
            pdl_trigger();
        }
        const uint4 now[kPieces][1] = {{tokens.v[0][0]}, {tokens.v[1][0]}};
        if (ahead.left != 0) {
            if (ahead.fresh) {
                tokens.rows(c, ahead.expert, 0, h, true, bytes);
                ahead.fresh = false;
            }
            tokens.load(ahead.step, bytes);
            ahead.advance();
        }
        if (lead == 1) {
            lead = 0;
            continue;
        }
        DownRing::wait();
        multiply<false>(acc, ring, now, false);
        ring.next();
        const int expert = walk.expert;
        if (walk.advance()) {
            down_add(a, c, sum, expert, acc);
            zero(acc);
        }
    }
    __syncthreads();
    if (blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll 1
    for (int v = tid; v < kDownRows * a.N; v += kLayerThreads) {
        float o = sums[v];
#pragma unroll 1
        for (int w = 1; w < kLayerWarps; ++w) o += sums[w * kDownRows * a.N + v];
        store_first(parts + rank * kDownRows * a.N + v, o);
    }
    // the first block joins the blocks' sums, in their order; nobody reads the others' memory
    if (blocks > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        if (rank != 0) return;
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
#pragma unroll 1
    for (int v = tid; v < kDownRows * a.N; v += kLayerThreads) {
        const int row = v % kDownRows, s = v / kDownRows;  // neighbouring threads write neighbouring elements
        if (row >= there) continue;
        float o = 0.f;
#pragma unroll 1
        for (uint32_t r = 0; r < blocks; ++r) o += parts[(r * kDownRows + row) * a.N + s];
        a.out[static_cast<int64_t>(s) * a.H + first_row + row] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
    }
}

}  // namespace moe

// ---------------------------------------------------------------- host
namespace {

using namespace moe_host;
using moe::LayerArgs;

// Blocks of these kernels that the GPU holds at once: two an SM by their threads and registers, one where the lists of
// many experts and pairs leave no room for two.  Grids have no more, as the rest would run after them, in a second wave
// (64 tokens, 8 of 384 experts of 2048 x 512: 357 us with two an SM, 345 with one; 8 tokens, 8 of 512: 80 and 75).
int resident_blocks(size_t smem) {
    constexpr size_t kOfAnSm = 228 * 1024, kOfTheSystem = 1024;  // of every block
    return num_sms() * (2 * (smem + kOfTheSystem) <= kOfAnSm ? 2 : 1);
}

template <bool Q, bool DOWN, int EIGHTS>
int launch_rows(const LayerArgs& a, cudaStream_t stream) {
    const size_t smem = moe::kLayerWarps * (moe::TileRing<DOWN>::kWarpBytes + sizeof(float4) * moe::kTiles * 32) +
                        moe::Chosen::bytes(a.N, a.K, a.E);
    if (cudaFuncSetAttribute(moe::layer_rows_kernel<Q, DOWN, EIGHTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(resident_blocks(smem))), block(moe::kLayerThreads);
    return launch(moe::layer_rows_kernel<Q, DOWN, EIGHTS>, grid, block, smem, stream, a);
}

int launch_down(const LayerArgs& a, cudaStream_t stream) {
    const size_t smem = moe::kLayerWarps * moe::DownRing::kWarpBytes +
                        sizeof(float) * (moe::kLayerWarps + moe::kDownBlocks) * moe::kDownRows * a.N +
                        moe::Chosen::bytes(a.N, a.K, a.E);
    if (cudaFuncSetAttribute(moe::layer_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess)
        return MOE_ERR_CUDA;
    // With so many rows that blocks alone fill the GPU, equal parts of them (above kDownRows a block there are more
    // blocks than the GPU holds); with fewer, as many blocks to a cluster as fit (a GPC's SMs are not all filled by
    // clusters, and one left for a second wave costs more than SMs with one block).
    const int slots = resident_blocks(smem);
    int rows = (a.H + slots - 1) / slots, blocks = 1;
    if (2 * rows <= moe::kDownRows) {
        rows = moe::kDownRows;
        while (blocks < moe::kDownBlocks && (a.H + rows - 1) / rows * blocks * 2 <= slots) blocks *= 2;
    }
    if (rows > moe::kDownRows) rows = moe::kDownRows;
    const int groups = (a.H + rows - 1) / rows;
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
    return cudaLaunchKernelEx(&cfg, moe::layer_down_kernel, a, rows) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace

extern "C" MOE_API size_t moe_layer_workspace_size(int N, int K, int H, int I) {
    if (N < 0 || N > MOE_LAYER_MAX_TOKENS || K < 1 || K > 32 || H < 8 || H % 8 != 0 || H >= 1 << 20 || I < 8 || I % 8 != 0 ||
        I >= 1 << 20)
        return 0;
    const size_t pairs = static_cast<size_t>(N > 0 ? N : 1) * K;
    return pairs * I * 2 + (N > moe::kDownTokens ? pairs * H * 4 : 0) + 2 * round16(pairs * 4);
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
    float* y = nullptr;
    if (N > 0 && K >= 1 && K <= 32) {
        if (workspace_bytes < moe_layer_workspace_size(N, K, H, I)) return MOE_ERR_CAPACITY;
        uint8_t* rest = static_cast<uint8_t*>(workspace) + static_cast<size_t>(N) * K * I * 2;
        y = reinterpret_cast<float*>(rest);
        if (N > moe::kDownTokens) rest += static_cast<size_t>(N) * K * H * 4;
        if (topk_idx == nullptr) topk_idx = reinterpret_cast<int32_t*>(rest);
        if (topk_w == nullptr) topk_w = reinterpret_cast<float*>(rest + round16(static_cast<size_t>(N) * K * 4));
    }
    // the router's own checks of logits, bias, E, K and its options come with its call
    const int rc = moe_route_topk(logits, bias, N, E, K, scoring, renormalize, n_group, topk_group, routed_scaling, topk_idx,
                                  topk_w, stream);
    if (rc != MOE_OK || N == 0) return rc;
    const LayerArgs a = {x, x_scale, w_gate_up, w_scale, w_down, topk_idx, topk_w, static_cast<uint16_t*>(workspace), y,
                         out, N, K, E, H, I};
    if (N <= moe::kDownTokens) {
        const int up = q ? launch_rows<true, false, 1>(a, stream) : launch_rows<false, false, 1>(a, stream);
        return up != MOE_OK ? up : launch_down(a, stream);
    }
    const int up = q ? launch_rows<true, false, 2>(a, stream) : launch_rows<false, false, 2>(a, stream);
    if (up != MOE_OK) return up;
    const int down = launch_rows<false, true, 2>(a, stream);
    if (down != MOE_OK) return down;
    const int64_t vecs = static_cast<int64_t>(N) * (H / 8);
    return launch(moe::layer_sum_kernel, dim3(static_cast<unsigned>((vecs + 255) / 256)), dim3(256), 0, stream, a);
}
