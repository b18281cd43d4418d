// expert_ffn.cu -- the experts' gated feed-forward over a plan's rows and
// its gradients (sm_103a).
//
// Five products, all grouped by expert (sum over k):
//   gated   g, u [row, i] = x[row, k] * w_gate_up[e][0|1][i][k]
//   down    y    [row, j] = h[row, k] * w_down[e][j][k]
//   dgate   dh   [row, i] = dy[row, k] * w_down[e][k][i]
//   dx      dx   [row, j] = dgate_up[row, k] * w_gate_up[e][k][j]
//   dw      dW[e][i][j]   = sum over the group's rows of left[row, i] * right[row, j]
// The forward call launches gated and down; the backward call dgate and, in
// one launch, dx and both weights' dw.
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
// halves to both SMs.  In the pair's first block warp 10 waits for the slices
// and warp 1 issues the matrix instructions.  Warps 2-9 read the accumulators (a warp sees 32 channels),
// turn them through shared memory so that a row's channels lie side by side,
// and write the output.  In the gated product every 32 rows of the M side are
// 16 channels of the gate and the same 16 of the up projection, so that a
// warp has both for silu(g) * u; dgate applies the activation's gradient to
// dh there, so that dh is never written.  dw's output rows are the
// accumulators' own: they leave by tensor copies of 32 rows by 64 columns.
//
// Where k is the contiguous index (x, h, dy, dgate_up; weights of gated and
// down) a stage holds rows of 64 k's (128 in 8 bits); where it is not (weights
// of dgate and dx, both sides of dw) it holds rows of 64 of the M or N index,
// one for each k, and the instruction reads it transposed.  Slices that leave
// an array are filled with zeros by the copy.  In dw a group's last slice runs
// on into other rows, which may hold anything: warp 11 of each block zeroes
// them in both operands as soon as the slice is there, while the instructions
// of the slices before it run.
//
// The pair's blocks agree on whether to run: the first one decides (see
// ffn_kernel).  A group without rows that has a place all the same gets one row
// tile without slices, for its padding's zeros.
//
// What bounds it, measured on a GB300 (6.68 TB/s copied, 1914 TFLOP/s in bf16
// at burst and 1721 under the power limit by the library): many rows, the tensor
// cores: 32768 rows, 8 experts, H = I = 4096: forward and backward 6.2 to 6.4 ms,
// 1550 to 1600 TFLOP/s, tensor pipes 70-87% busy (gated in 8 bits, 8192 rows
// profiled alone: 3.4 PFLOP/s).  Few rows, the weights' bytes: 61 tokens over 64 experts of 4096 x 1280,
// 212 us, 6.3 TB/s of what has to be read.  One token through 8 experts of
// 2048 x 768, 26 us: 10 and 5 of them stream the weights, the rest are the two
// launches' fixed costs.
#include <cuda_fp8.h>

#include "tensor_core.cuh"
#include "vec8.cuh"

namespace moe {

enum Product { kGated, kDown, kDgate, kDx, kDw, kGrads };  // kGrads: dx and two dw

constexpr int kTile = 256;         // both sides of a tile at most
constexpr int kHalf = 128;         // a block's part of it
constexpr int kSlice = 128;        // bytes of a stage's row
constexpr int kMaxStages = 12;
constexpr int kEpilogueWarps = 8;
constexpr int kWatchWarp = 2 + kEpilogueWarps;
constexpr int kMendWarp = kWatchWarp + 1;  // of launches with dw
constexpr int kOrders = 16;        // tiles whose orders are kept: more than slices that can be ready
constexpr int kRun = 1, kStop = 2;  // Shared::decision
constexpr int kChunk = 16;         // accumulator columns that a warp turns at a time

__host__ __device__ constexpr int ffn_threads(int p) { return 96 + 32 * kEpilogueWarps + (p == kGrads ? 32 : 0); }
// a warp's bytes to turn a chunk in: dw sends boxes of 4 KB, which start at multiples of 1024 (they are swizzled)
__host__ __device__ constexpr int ffn_turn(int p) { return p == kGrads ? 4096 : 2048; }
__host__ __device__ constexpr int ffn_jobs(int p) { return p == kGrads ? 3 : 1; }

struct Job {
    CUtensorMap map_m;
    CUtensorMap map_n[5];   // the N side by 16, 32, 64, 96 and 128 rows (dw: [0], by columns)
    CUtensorMap map_out;    // dw: the output
    int M, N, K;            // M: output channels; K: contraction length; dw: output M x N; M = 0: no work
    int m_whole, n_whole;   // a block's part of a slice is one copy (see make_job)
    uint16_t* out;
};

struct Common {
    const float* a_scale;   // gated in 8 bits: scales of x's rows and of the channels
    const float* b_scale;
    const float* preact_in;
    float* preact_out;
    const int32_t* cu;
    const int32_t* count;
    int32_t* status;
    int64_t rows;
    int E;
    int ring_bytes;
    int early;              // a call's second or later kernel
    int64_t timeout_ns;
};

template <int P>
struct Launch {
    Job job[ffn_jobs(P)];
    Common c;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], tail_full[kMaxStages], tail_ready[kMaxStages], acc_full[2],
        acc_empty[2];
    uint4 order[kOrders];   // the tiles' instructions: descriptor, slices (0: the end), steps of the last, dw
    uint32_t ready;         // slices that the instructions may use, counted from the launch's start
    uint32_t tmem;
    int stop;               // the plan's status held an error when this block read it
    int decision;           // in the pair's second block: what the first one decided
    int started;            // the kernel ahead has ended
    int failed;             // a wait of this block ran out
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

// The groups, as every warp of a block sees them.
struct Groups {
    const int *first, *count, *padded;
    const int* prefix;  // row tiles before each expert [E + 1]
    int E;
};

// A group's row tiles; one without rows has one for its padding's zeros.
__device__ __forceinline__ int group_tiles(int count, int padded) {
    return count > 0 ? (count + kTile - 1) / kTile : padded > 0 ? 1 : 0;
}

// A product's tiles in order: expert by expert, and within one in bands of 8
// tiles of the N side with the M side outermost, so that what the pairs work
// on at one time is about square and stays in L2.  A warp walks over its own
// tiles (each as many as there are pairs after the last), all lanes together:
// the next expert is found by a vote over 32 at a time, since a search by one
// thread (some 2000 cycles with its divisions) left the tensor cores without
// work between tiles.  Spreading experts of few rows among those of many, to
// mix tiles bound by memory with tiles bound by the products, was measured and
// is slower (2009 against 1930 us a step at 65536 rows, 128 experts, Zipf).
template <int P, bool FP8>
struct Tiles {
    int m_step, m_tiles, n_tiles, k_slices, N;
    int64_t each, total;    // tiles of a row tile (dw: of an expert), and of all
    int e = 0, nt = 0, length = 0;
    int64_t begin = 0, end = 0;  // the current expert's tiles

    __device__ __forceinline__ Tiles(const Job& j, const Groups& g) {
        m_step = P == kGated ? kHalf : kTile;  // a gated tile holds each channel twice
        m_tiles = (j.M + m_step - 1) / m_step;
        n_tiles = P == kDw ? (j.N + kTile - 1) / kTile : 0;
        N = j.N;
        k_slices = (j.K + (FP8 ? 127 : 63)) / (FP8 ? 128 : 64);
        each = P == kDw ? static_cast<int64_t>(m_tiles) * n_tiles : m_tiles;
        total = each * (P == kDw ? g.E : g.prefix[g.E]);
    }

    // Tile i < total, not before the one asked for last; all lanes of a warp.
    __device__ __forceinline__ Tile at(const Groups& g, int64_t i, int lane) {
        if (i >= end) {
            if constexpr (P == kDw) {
                e = static_cast<int>(i / each);
                begin = e * each;
                end = begin + each;
                nt = n_tiles;
            } else {
                while (true) {  // the first expert whose tiles end past i
                    const int mine = min(e + 1 + lane, g.E);
                    const uint32_t past = __ballot_sync(FULL_MASK, g.prefix[mine] * each > i);
                    if (past != 0) {
                        e += __ffs(static_cast<int>(past)) - 1;
                        break;
                    }
                    e += 32;
                }
                begin = g.prefix[e] * each;
                end = g.prefix[e + 1] * each;
                nt = g.prefix[e + 1] - g.prefix[e];
                length = ((g.count[e] + nt - 1) / nt + 15) & ~15;
            }
        }
        Tile r;
        r.e = e;
        r.first = g.first[e];
        r.count = g.count[e];
        r.padded = g.padded[e];
        constexpr int kBand = 8;
        int rest = static_cast<int>(i - begin), j = 0;
        if (nt > kBand) {
            const int band = rest / (kBand * m_tiles);
            j = band * kBand;
            rest -= j * m_tiles;
        }
        const int width = min(kBand, nt - j), m = rest / width;
        r.m0 = m * m_step;
        j += rest - m * width;
        r.last = j == nt - 1;
        if constexpr (P == kDw) {
            r.n0 = j * kTile;
            r.n = min(kTile, N - r.n0);
            r.slices = (r.count + 63) / 64;
        } else {
            r.n0 = j * length;
            r.n = min(length, r.count - r.n0);
            r.slices = r.n > 0 ? k_slices : 0;
        }
        return r;
    }
};

// Where a pair is in a launch's tiles, over all its jobs.
struct Turn {
    int64_t next;   // its next tile, counted from the first one of the current job
    int pairs;
};

// Bounded wait; on a timeout the caller gives up and the plan's status says so.
// It also gives up where the pair's first block has stopped.  The limit is for a
// slice's steps.  A wait that lasts for many slices, a whole tile's or more, gets
// a 65536th of it for each (15 us of the usual second, where a slice takes 0.3 to
// 0.8).  Its clock does not run while the kernel ahead still does.  All but the
// first test stays out of line: inlined at every wait it cost 0.6 us a call.
__device__ __noinline__ bool wait_on(int64_t timeout_ns, int32_t* status, const Shared* sh, const uint64_t* bar,
                                     uint32_t parity, uint64_t slices) {
    const volatile Shared* v = sh;
    const uint64_t limit = static_cast<uint64_t>(timeout_ns) + static_cast<uint64_t>(timeout_ns >> 16) * slices;
    uint64_t t0 = 0;
    do {
        if (v->decision == kStop) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0 || v->started == 0) {
            t0 = now;
        } else if (now - t0 > limit) {
            record_error(status, MOE_ERR_DEVICE_TIMEOUT, blockIdx.x);
            return false;
        }
    } while (!mbar_try_pair(bar, parity));
    return true;
}
__device__ __forceinline__ bool wait(const Common& c, const Shared* sh, const uint64_t* bar, uint32_t parity,
                                     uint64_t slices = 0) {
    return mbar_try_pair(bar, parity) || wait_on(c.timeout_ns, c.status, sh, bar, parity, slices);
}

template <int P>
__host__ __device__ constexpr bool m_transposed() { return P == kDgate || P == kDx || P == kDw; }
template <int P>
__host__ __device__ constexpr bool n_transposed() { return P == kDw; }

struct RingShape {
    uint8_t* at;
    uint32_t stage_bytes;
    int stages;
};

// ---------------------------------------------------------------- copies in (a warp of each block, one lane)
struct Producer {
    Turn turn;
    int s = 0;
    uint32_t phase = 0;
    int ahead = 0;           // slices of the first tile whose M side is on its way already
    bool ok = true;

    // The N side of a block's part of a tile: its rows, brought by one copy of
    // 16 or a multiple of 32 of them (dw: columns, by one copy of 128 or by
    // copies of 64).
    struct NSide {
        int rows, piece, pieces;
        uint32_t bytes;      // of a block's part of a slice, both sides
    };
    template <int P>
    __device__ __forceinline__ NSide n_side(const Job& job, const Tile& t) const {
        NSide n;
        n.rows = ((t.n + 15) & ~15) / 2;
        n.piece = P == kDw ? (job.n_whole ? 128 : 64) : n.rows > 16 ? (n.rows + 31) & ~31 : 16;
        n.pieces = P == kDw ? (n.rows + n.piece - 1) / n.piece : 1;
        n.bytes = static_cast<uint32_t>(kHalf + n.pieces * n.piece) * kSlice;
        return n;
    }

    // Where a tile's copies come from: the coordinates that stay for all its slices.
    struct Source {
        int m, e, first;     // M side: channel, expert; dw: the group's first row
        int n;               // N side: first row (dw: column)
        const CUtensorMap* map_n;
        NSide side;
    };
    template <int P>
    __device__ __forceinline__ Source source(const Job& job, const Tile& t, int rank) const {
        Source f;
        f.side = n_side<P>(job, t);
        f.m = t.m0 + rank * (P == kGated ? 64 : kHalf);
        f.e = t.e;
        f.first = t.first;
        f.n = (P == kDw ? t.n0 : t.first + t.n0) + rank * f.side.rows;
        f.map_n = &job.map_n[P == kDw ? 0 : f.side.piece / 32];
        return f;
    }
    // A block's part of the slice that starts at k.
    template <int P>
    static __device__ __forceinline__ void copy_m(const Job& job, const Source& f, int k, uint32_t to, uint32_t bar) {
        if constexpr (P == kGated) {
            if (job.m_whole) tensor_load_5d(to, &job.map_m, k, 0, 0, f.m / 16, f.e, bar);
            else
                for (int j = 0; j < 4; ++j) tensor_load_4d(to + j * 4096, &job.map_m, k, f.m + 16 * j, 0, f.e, bar);
        } else if constexpr (P == kDown) {
            tensor_load_3d(to, &job.map_m, k, f.m, f.e, bar);
        } else if constexpr (P == kDw) {
            if (job.m_whole) tensor_load_3d(to, &job.map_m, 0, f.first + k, f.m / 64, bar);
            else
                for (int j = 0; j < 2; ++j) tensor_load_2d(to + j * 8192, &job.map_m, f.m + 64 * j, f.first + k, bar);
        } else {
            if (job.m_whole) tensor_load_4d(to, &job.map_m, 0, k, f.m / 64, f.e, bar);
            else
                for (int j = 0; j < 2; ++j) tensor_load_3d(to + j * 8192, &job.map_m, f.m + 64 * j, k, f.e, bar);
        }
    }
    template <int P>
    static __device__ __forceinline__ void copy_n(const Job& job, const Source& f, int k, uint32_t to, uint32_t bar) {
        if constexpr (P == kDw) {
            if (job.n_whole) tensor_load_3d(to, f.map_n, 0, f.first + k, f.n / 64, bar);
            else
                for (int j = 0; j < f.side.pieces; ++j) tensor_load_2d(to + j * 8192, f.map_n, f.n + 64 * j, f.first + k, bar);
        } else {
            tensor_load_2d(to, f.map_n, k, f.n, bar);
        }
    }

    // The M side (weights) of the first tile's first slices, before the rows are there.
    template <int P, bool FP8>
    __device__ __forceinline__ void start(const Job& job, const Groups& g, Shared* sh, const RingShape& ring, int rank,
                                          int lane) {
        Tiles<P, FP8> tiles(job, g);
        if (turn.next >= tiles.total) return;
        const Tile t = tiles.at(g, turn.next, lane);
        const Source f = source<P>(job, t, rank);
        ahead = min(ring.stages, t.slices);
        if (lane == 0)
            for (int k = 0; k < ahead; ++k) {
                const uint32_t bar = rank == 0 ? smem_addr(&sh->full[k]) : leader_addr(&sh->full[k]);
                if (rank == 0) mbar_expect(bar, 2 * f.side.bytes);
                copy_m<P>(job, f, k * (FP8 ? 128 : 64), smem_addr(ring.at + k * ring.stage_bytes), bar);
            }
    }

    template <int P, bool FP8>
    __device__ __forceinline__ void run(const Job& job, const Common& c, const Groups& g, Shared* sh,
                                        const RingShape& ring, int rank, int lane) {
        constexpr int kElems = FP8 ? 128 : 64;
        Tiles<P, FP8> tiles(job, g);
        const uint32_t base = smem_addr(ring.at);
        const uint32_t full = rank == 0 ? smem_addr(&sh->full[0]) : leader_addr(&sh->full[0]);
        for (; ok && turn.next < tiles.total; turn.next += turn.pairs) {
            const Tile t = tiles.at(g, turn.next, lane);
            const Source f = source<P>(job, t, rank);
            // Both blocks' copies are counted by the first one's barrier, but those
            // of a slice that has to be mended by each block's own.
            const int mended = P == kDw && (t.count & 15) != 0 ? t.slices - 1 : -1;
            for (int k = 0; k < t.slices && lane == 0; ++k) {
                const uint32_t to = base + static_cast<uint32_t>(s) * ring.stage_bytes;
                uint32_t bar = full + 8u * static_cast<uint32_t>(s);
                if (ahead > 0) {
                    --ahead;
                } else {
                    if (!(ok = wait(c, sh, &sh->empty[s], phase ^ 1u))) break;
                    if (P == kDw && k == mended) {
                        bar = smem_addr(&sh->tail_full[s]);
                        mbar_expect(bar, f.side.bytes);
                    } else if (rank == 0) {
                        mbar_expect(bar, 2 * f.side.bytes);
                    }
                    copy_m<P>(job, f, k * kElems, to, bar);
                }
                copy_n<P>(job, f, k * kElems, to + kHalf * kSlice, bar);
                if (++s == ring.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            __syncwarp();
            ok = __shfl_sync(FULL_MASK, static_cast<int>(ok), 0) != 0;
        }
        turn.next -= tiles.total;
    }
};

// ---------------------------------------------------------------- matrix instructions (two warps of the pair's first block)
// A barrier's test between matrix instructions costs the thread that issues
// them some 190 cycles even where the barrier is long complete (measured: 4
// instructions and a commit take 270 cycles for N <= 64, 385 for N = 192, 513
// for N = 256; with a test 458, 458, 513).  So another warp does all the
// waiting: it walks over the tiles, leaves each one's orders in shared memory,
// waits for its slices and counts those that are ready.  The issuing thread
// reads the count, and only when it has used up what it read last.
struct Watcher {
    Turn turn;
    int s = 0, buf = 0;
    uint32_t acc_phase = 0, full_phase = 0, tail_phase = 0;  // the latter two: a bit a stage
    uint32_t slices = 0, tiles_seen = 0;
    bool ok = true;

    __device__ __forceinline__ void publish(Shared* sh, int lane) {
        ++slices;
        if (lane == 0)
            asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_addr(&sh->ready)), "r"(slices) : "memory");
    }

    template <int P, bool FP8>
    __device__ __forceinline__ void run(const Job& job, const Common& c, const Groups& g, Shared* sh, int stages,
                                        int lane) {
        Tiles<P, FP8> tiles(job, g);
        for (; ok && turn.next < tiles.total; turn.next += turn.pairs) {
            const Tile t = tiles.at(g, turn.next, lane);
            if (t.slices == 0) continue;
            const bool tail = P == kDw && (t.count & 15) != 0;
            if (lane == 0)
                sh->order[tiles_seen % kOrders] =
                    make_uint4(mma_desc(FP8 ? 0u : 1u, m_transposed<P>(), n_transposed<P>(), kTile, (t.n + 15) & ~15),
                               t.slices, P == kDw ? ((t.count - 1) % 64) / 16 + 1 : 4, P == kDw);
            ++tiles_seen;
            ok = __all_sync(FULL_MASK, wait(c, sh, &sh->acc_empty[buf], acc_phase ^ 1u));
            for (int k = 0; k < t.slices && ok; ++k) {
                if (tail && k + 1 == t.slices) {
                    ok = __all_sync(FULL_MASK, wait(c, sh, &sh->tail_ready[s], (tail_phase >> s) & 1u));
                    tail_phase ^= 1u << s;
                } else {
                    ok = __all_sync(FULL_MASK, wait(c, sh, &sh->full[s], (full_phase >> s) & 1u));
                    full_phase ^= 1u << s;
                }
                if (ok) publish(sh, lane);
                if (++s == stages) s = 0;
            }
            if ((buf ^= 1) == 0) acc_phase ^= 1u;
        }
        turn.next -= tiles.total;
    }

    // After the last job, or after a wait that ran out: nothing comes any more.
    __device__ __forceinline__ void end(Shared* sh, int lane) {
        if (lane == 0) sh->order[tiles_seen % kOrders] = make_uint4(0u, 0u, 0u, 0u);
        publish(sh, lane);
    }
};

struct Issuer {
    int s = 0, buf = 0;
    uint32_t used = 0, ready = 0;
    bool ok = true;

    // Whether slice `used` is there; gives up after as long as any wait does.
    __device__ __forceinline__ bool more(const Common& c, Shared* sh) {
        if (used != ready) return true;
        uint64_t t0 = 0;
        for (uint32_t n = 0;; ++n) {
            asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(ready) : "r"(smem_addr(&sh->ready)) : "memory");
            if (used != ready) break;
            if ((n & 255u) == 255u) {
                const uint64_t now = globaltimer_ns();
                if (t0 == 0 || static_cast<const volatile Shared*>(sh)->started == 0) t0 = now;
                else if (now - t0 > 2 * static_cast<uint64_t>(c.timeout_ns)) return ok = false;  // the watcher's limit first
            }
        }
        tc_fence_after();
        return true;
    }

    template <int P, bool FP8>
    __device__ __forceinline__ void tile(const Common& c, Shared* sh, const RingShape& ring, uint32_t tmem,
                                         const uint4& order) {
        constexpr bool kMt = m_transposed<P>(), kNt = n_transposed<P>();
        constexpr int kStepM = (kMt ? 2048 : 32) >> 4, kStepN = (kNt ? 2048 : 32) >> 4;
        const uint32_t acc = tmem + buf * kTile, desc = order.x;
        for (uint32_t k = 0; k < order.y; ++k) {
            if (!more(c, sh)) return;
            const bool last = k + 1 == order.y;
            const uint32_t sm = smem_addr(ring.at + s * ring.stage_bytes);
            const uint64_t dm = operand_desc(sm, kMt ? 8192 : 16, 1024);
            const uint64_t dn = operand_desc(sm + kHalf * kSlice, kNt ? 8192 : 16, 1024);
            // 32 bytes of k, or 16 rows of it, an instruction; dw's last slice may have fewer
            if (P != kDw || !last || order.z == 4u) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mma<FP8>(acc, dm + j * kStepM, dn + j * kStepN, desc, k > 0 || j > 0);
            } else {
                for (uint32_t j = 0; j < order.z; ++j)
                    mma<FP8>(acc, dm + j * kStepM, dn + j * kStepN, desc, k > 0 || j > 0);
            }
            mma_commit(&sh->empty[s]);
            if (last) mma_commit(&sh->acc_full[buf]);
            if (++s == ring.stages) s = 0;
            ++used;
        }
        buf ^= 1;
    }

    template <int P, bool FP8>
    __device__ __forceinline__ void run(const Common& c, Shared* sh, const RingShape& ring, uint32_t tmem) {
        for (uint32_t i = 0; ok && more(c, sh); ++i) {
            const uint4 order = sh->order[i % kOrders];
            if (order.y == 0) break;
            if (P == kGrads && order.w != 0) tile<kDw, false>(c, sh, ring, tmem, order);
            else tile<P == kGrads ? kDx : P, FP8>(c, sh, ring, tmem, order);
        }
    }
};

// ---------------------------------------------------------------- dw's last slices (a warp of each block)
struct Mender {
    Turn turn;
    int s = 0;
    uint32_t tail_phase = 0;
    uint64_t passed = 0;     // slices since the last one waited for
    bool ok = true;

    template <int P>
    __device__ __forceinline__ void run(const Job& job, const Common& c, const Groups& g, Shared* sh,
                                        const RingShape& ring, int lane) {
        Tiles<P, false> tiles(job, g);
        for (; ok && turn.next < tiles.total; turn.next += turn.pairs) {
            const Tile t = tiles.at(g, turn.next, lane);
            if (t.slices == 0) continue;
            if (P != kDw) {  // only to know where in the ring the next job starts
                s = (s + t.slices) % ring.stages;
                passed += t.slices;
                continue;
            }
            s = (s + t.slices - 1) % ring.stages;
            passed += t.slices;
            if ((t.count & 15) != 0) {
                ok = __all_sync(FULL_MASK, wait(c, sh, &sh->tail_full[s], (tail_phase >> s) & 1u, passed));
                if (!ok) break;
                passed = 0;
                tail_phase ^= 1u << s;
                // rows from the group's end to a multiple of 16; the N side's boxes of
                // 64 columns follow the M side's two in the stage
                const int valid = t.count & 63, chunks = (((valid + 15) & ~15) - valid) * 8;
                const int boxes = 2 + (((t.n + 15) & ~15) / 2 + 63) / 64;
                uint8_t* at = ring.at + s * ring.stage_bytes + valid * kSlice;
                for (int j = lane; j < boxes * chunks; j += 32)
                    *reinterpret_cast<uint4*>(at + j / chunks * 8192 + j % chunks * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(&sh->tail_ready[s]);
            }
            if (++s == ring.stages) s = 0;
        }
        turn.next -= tiles.total;
    }
};

// ---------------------------------------------------------------- output (eight warps of each block)
// sigmoid(g) and 1 - sigmoid(g) from e = exp(-|g|), which neither overflows nor
// takes the division's divisor beyond 2.  __expf is documented to within
// 2 + floor(1.173 |g|) units in the last place, __fdividef to within 2: for
// |g| < 16 less than 23 units in all, under 2^-18.4 relative, and for any g under
// |g| * 2^-22 and a few units, until e leaves the normal numbers at |g| > 87.3.
struct Sigmoid {
    float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float g) {
    const float e = __expf(-fabsf(g)), near = __fdividef(1.f, 1.f + e), far = e * near;
    return g < 0.f ? Sigmoid{far, near} : Sigmoid{near, far};
}
__device__ __forceinline__ float silu(float g) { return g * sigmoid(g).s; }

__device__ __forceinline__ void store4_bf16(uint16_t* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(a, b), pack2(c, d));
}

// dgate: the pre-activations that a lane needs for a chunk.  Gated in 8 bits:
// the scales of its four channels (g[0], u[0]).
struct Saved {
    float4 g[kChunk / 4], u[kChunk / 4];
};
__device__ __forceinline__ void load_saved(Saved& s, const Job& job, const Common& a, const Tile& t, int rank, int c0,
                                           int quarter, int lane) {
    const int64_t M = job.M;
    const int c = t.m0 + rank * kHalf + quarter * 32 + (lane & 7) * 4;
#pragma unroll
    for (int it = 0; it < kChunk / 4; ++it) {
        const int n = c0 + it * 4 + (lane >> 3);
        if (n < t.n && c < M) {
            const float* pre = a.preact_in + (t.first + static_cast<int64_t>(t.n0 + n)) * 2 * M + c;
            s.g[it] = ld_stream_f4(pre);
            s.u[it] = ld_stream_f4(pre + M);
        }
    }
}

// One chunk of a row product: 16 rows of the group by the warp's 32 channels,
// turned through `turn` [16][32] so that neighbouring lanes hold neighbouring
// channels.  Odd rows have their halves swapped: the gated product reads two
// rows' same half at a time.
template <int P, bool FP8>
__device__ __forceinline__ void epilogue_chunk(const Job& job, const Common& a, const Tile& t, int rank, uint32_t acc,
                                               int c0, int quarter, int lane, float* turn, const Saved& saved) {
    const int64_t M = job.M;
    uint32_t v[kChunk];
    auto turned = [&](int j, int c) { return reinterpret_cast<float4*>(turn + j * 32 + (c ^ ((j & 1) << 4))); };
    auto turn_in = [&] {
        __syncwarp();
        tmem_load16(acc + c0, v);
        tmem_wait_load();
#pragma unroll
        for (int j = 0; j < kChunk; ++j) turn[j * 32 + (lane ^ ((j & 1) << 4))] = __uint_as_float(v[j]);
        __syncwarp();
    };
    if constexpr (P == kGated) {
        const int c = t.m0 + rank * 64 + quarter * 16 + (lane & 3) * 4;  // this lane's 4 channels
        turn_in();
#pragma unroll
        for (int it = 0; it < kChunk / 8; ++it) {
            const int j = it * 8 + (lane >> 2), n = c0 + j;
            if (n >= t.n || c >= M) continue;
            const int64_t row = t.first + static_cast<int64_t>(t.n0 + n);
            float4 g = *turned(j, (lane & 3) * 4);
            float4 u = *turned(j, 16 + (lane & 3) * 4);
            if constexpr (FP8) {
                const float s = __ldg(a.a_scale + row);
                const float4 sg = saved.g[0], su = saved.u[0];
                g = make_float4(g.x * (s * sg.x), g.y * (s * sg.y), g.z * (s * sg.z), g.w * (s * sg.w));
                u = make_float4(u.x * (s * su.x), u.y * (s * su.y), u.z * (s * su.z), u.w * (s * su.w));
            }
            if (a.preact_out != nullptr) {
                *reinterpret_cast<float4*>(a.preact_out + row * 2 * M + c) = g;
                *reinterpret_cast<float4*>(a.preact_out + row * 2 * M + M + c) = u;
            }
            store4_bf16(job.out + row * M + c, silu(g.x) * u.x, silu(g.y) * u.y, silu(g.z) * u.z, silu(g.w) * u.w);
        }
    } else {
        const int c = t.m0 + rank * kHalf + quarter * 32 + (lane & 7) * 4;
        constexpr int kIts = kChunk / 4;
        turn_in();
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
            const int j = it * 4 + (lane >> 3), n = c0 + j;
            if (n >= t.n || c >= M) continue;
            const int64_t row = t.first + static_cast<int64_t>(t.n0 + n);
            const float4 d = *turned(j, (lane & 7) * 4);
            if constexpr (P == kDgate) {
                const float dh[4] = {d.x, d.y, d.z, d.w}, gs[4] = {saved.g[it].x, saved.g[it].y, saved.g[it].z, saved.g[it].w},
                            us[4] = {saved.u[it].x, saved.u[it].y, saved.u[it].z, saved.u[it].w};
                float dg[4], du[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const Sigmoid s = sigmoid(gs[i]);
                    dg[i] = dh[i] * us[i] * s.s * fmaf(gs[i], s.rest, 1.f);
                    du[i] = dh[i] * gs[i] * s.s;
                }
                store4_bf16(job.out + row * 2 * M + c, dg[0], dg[1], dg[2], dg[3]);
                store4_bf16(job.out + row * 2 * M + M + c, du[0], du[1], du[2], du[3]);
            } else {
                store4_bf16(job.out + row * M + c, d.x, d.y, d.z, d.w);
            }
        }
    }
}

// dw: 64 columns of the warp's 32 rows, written to `box` as the tensor copy
// wants them (rows of 128 bytes, 16-byte pieces swizzled) and sent off.
__device__ __forceinline__ void epilogue_dw(const Job& job, const Tile& t, int rank, uint32_t acc, int c0, int quarter,
                                            int lane, uint4* box) {
    const int m = t.m0 + rank * kHalf + quarter * 32;
    if (lane == 0) bulk_wait_read<0>();  // the box before has left
    __syncwarp();
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        uint32_t v[2][16];
        if (t.slices > 0) {
            tmem_load16(acc + c0 + 32 * part, v[0]);
            tmem_load16(acc + c0 + 32 * part + 16, v[1]);
            tmem_wait_load();
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j / 16][j % 16] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t* f = v[q / 2] + 8 * (q & 1);
            uint32_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = pack2(__uint_as_float(f[2 * j]), __uint_as_float(f[2 * j + 1]));
            box[lane * 8 + ((4 * part + q) ^ (lane & 7))] = make_uint4(p[0], p[1], p[2], p[3]);
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && m < job.M) {
        tensor_store_3d(&job.map_out, t.n0 + c0, m, t.e, box);
        bulk_commit();
    }
}

struct Drain {
    Turn turn;
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;

    template <int P, bool FP8>
    __device__ __forceinline__ void run(const Job& job, const Common& c, const Groups& g, Shared* sh, uint32_t tmem,
                                        int rank, int warp, int lane, uint8_t* turn_buf) {
        const int quarter = warp & 3;           // the lanes of tensor memory that a warp may read
        const int half = (warp - 2) >> 2;       // two warps a quarter take every other chunk
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        Tiles<P, FP8> tiles(job, g);
        for (; ok && turn.next < tiles.total; turn.next += turn.pairs) {
            const Tile t = tiles.at(g, turn.next, lane);
            Saved now, next;  // dgate: asked for before the products are done, and a chunk ahead
            if constexpr (P == kDgate) load_saved(now, job, c, t, rank, half * kChunk, quarter, lane);
            if constexpr (P == kGated && FP8) {
                const int channel = t.m0 + rank * 64 + quarter * 16 + (lane & 3) * 4;
                if (channel < job.M) {
                    const float* scale = c.b_scale + 2 * static_cast<int64_t>(job.M) * t.e + channel;
                    now.g[0] = __ldg(reinterpret_cast<const float4*>(scale));
                    now.u[0] = __ldg(reinterpret_cast<const float4*>(scale + job.M));
                }
            }
            if (t.slices > 0) {
                ok = __all_sync(FULL_MASK, wait(c, sh, &sh->acc_full[buf], acc_phase, t.slices));
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t acc = tmem + buf * kTile + lanes;
            if constexpr (P == kDw) {
                for (int n = half * 64; n < t.n; n += 128) epilogue_dw(job, t, rank, acc, n, quarter, lane, reinterpret_cast<uint4*>(turn_buf));
            } else {
                for (int n = half * kChunk; n < t.n; n += 2 * kChunk) {
                    if constexpr (P == kDgate) load_saved(next, job, c, t, rank, n + 2 * kChunk, quarter, lane);
                    epilogue_chunk<P, FP8>(job, c, t, rank, acc, n, quarter, lane, reinterpret_cast<float*>(turn_buf), now);
                    if constexpr (P == kDgate) now = next;
                }
            }
            if (t.slices > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(&sh->acc_empty[buf]);
                if ((buf ^= 1) == 0) acc_phase ^= 1u;
            }
            if constexpr (P == kDown || P == kDx) {  // the group's padding: zeros
                if (t.last && t.padded > t.count) {
                    const int c0 = t.m0 + rank * kHalf, chunks = (min(kHalf, job.M - c0) + 7) / 8;
                    const int64_t todo = chunks > 0 ? static_cast<int64_t>(t.padded - t.count) * chunks : 0;
                    for (int64_t j = (warp - 2) * 32 + lane; j < todo; j += 32 * kEpilogueWarps)
                        st_v4(job.out + (t.first + t.count + j / chunks) * static_cast<int64_t>(job.M) + c0 +
                                  8 * (j % chunks),
                              make_uint4(0u, 0u, 0u, 0u));
                }
            }
        }
        turn.next -= tiles.total;
    }
};

// ---------------------------------------------------------------- the kernel
template <int P, bool FP8>
__global__ void __launch_bounds__(ffn_threads(P), 1) ffn_kernel(const __grid_constant__ Launch<P> a) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int kThreads = ffn_threads(P), kWarps = kThreads / 32;
    const Common& c = a.c;
    uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* turns = base + c.ring_bytes;
    Shared* sh = reinterpret_cast<Shared*>(turns + kEpilogueWarps * ffn_turn(P));
    const int E = c.E;
    int* first = reinterpret_cast<int*>(sh + 1);
    int *count = first + E, *padded = count + E, *prefix = padded + E;  // prefix: E + 1

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(pair_rank());
    if (tid == 0) {
        if (a.job[0].M > 0) {  // else its maps are not set
            tensor_prefetch(&a.job[0].map_m);
            tensor_prefetch(&a.job[0].map_n[4]);
        }
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
        sh->ready = 0;
        sh->decision = 0;
        sh->started = !c.early;
        sh->failed = 0;
    }
    __syncwarp();
    if (warp == 1) tmem_alloc(&sh->tmem, 512);
    tc_fence_before();
    __syncwarp();
    pair_arrive();  // this warp's part of the block is set up; the wait comes after the groups' scan
    // A call's later kernels start while the one before still runs: the groups
    // and the weights were there before that one began, and only the warps that
    // touch the rows wait for it.
    if (!c.early) {
        pdl_wait();
        pdl_trigger();
    }
    if (tid == 0) sh->stop = ld_volatile_s32(c.status) != 0;

    // ---- the groups: row tiles before each expert
    const int per = (E + kThreads - 1) / kThreads;
    int mine = 0, longest = 0;
    for (int e = tid * per; e < min(E, (tid + 1) * per); ++e) {
        const int64_t f = __ldg(c.cu + e), n = __ldg(c.count + e), after = __ldg(c.cu + e + 1);
        const int64_t p = after - f;
        const bool fits = n >= 0 && f >= 0 && p >= n && f + p <= c.rows;
        if (!fits) record_error(c.status, MOE_ERR_DEVICE_INDEX, e);
        first[e] = fits ? static_cast<int>(f) : 0;
        count[e] = fits ? static_cast<int>(n) : 0;
        padded[e] = fits ? static_cast<int>(p) : 0;
        mine += group_tiles(count[e], padded[e]);
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
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += sh->scan[i];
        row_tiles += sh->scan[i];
        longest = max(longest, sh->most[i]);
    }
    for (int e = tid * per; e < min(E, (tid + 1) * per); ++e) {
        prefix[e] = before;
        before += group_tiles(count[e], padded[e]);
    }
    if (tid == 0) prefix[E] = row_tiles;
    const Groups g = {first, count, padded, prefix, E};
    // short groups leave room for more stages: the N side's part is as long as the longest tile's half
    const int half = (min(longest, kTile) + 15) / 16 * 8;
    const int n_rows = P == kGrads ? kHalf : half > 16 ? (half + 31) / 32 * 32 : 16;
    RingShape ring;
    ring.at = base;
    ring.stage_bytes = static_cast<uint32_t>(kHalf + n_rows) * kSlice;
    ring.stages = min(kMaxStages, static_cast<int>(c.ring_bytes / ring.stage_bytes));
    Turn turn;
    turn.next = blockIdx.x >> 1;
    turn.pairs = static_cast<int>(gridDim.x >> 1);
    __syncthreads();
    pair_wait();  // both blocks' barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    // The pair's first block decides for both whether there is an error already:
    // other blocks may record one between the two reads. The second block does
    // not wait for the decision (that cost a launch 0.4 us) unless it has
    // read an error itself: once it works, its waits look for it.
    bool run = sh->stop == 0;
    if (rank == 0) {
        if (tid == 0) set_in_second(&sh->decision, run ? kRun : kStop);
    } else if (!run) {
        const uint64_t t0 = globaltimer_ns();
        while (*static_cast<volatile int*>(&sh->decision) == 0)
            if (globaltimer_ns() - t0 > static_cast<uint64_t>(c.timeout_ns)) break;
        run = *static_cast<volatile int*>(&sh->decision) == kRun;
    }
    if (!run && c.early) pdl_wait();

    if (run && warp == 0) {
        Producer r;
        r.turn = turn;
        if (c.early) {
            if constexpr (P == kDown) r.start<P, FP8>(a.job[0], g, sh, ring, rank, lane);
            if constexpr (P == kGrads)
                if (a.job[0].M > 0) r.start<kDx, false>(a.job[0], g, sh, ring, rank, lane);
            __syncwarp();
            pdl_wait();
            pdl_trigger();
            if (lane == 0) static_cast<volatile Shared*>(sh)->started = 1;
        }
        if constexpr (P == kGrads) {
            if (a.job[0].M > 0) r.run<kDx, false>(a.job[0], c, g, sh, ring, rank, lane);
            if (a.job[1].M > 0) r.run<kDw, false>(a.job[1], c, g, sh, ring, rank, lane);
            if (a.job[2].M > 0) r.run<kDw, false>(a.job[2], c, g, sh, ring, rank, lane);
        } else {
            r.run<P, FP8>(a.job[0], c, g, sh, ring, rank, lane);
        }
        if (!r.ok) sh->failed = 1;
    } else if (run && warp == 1 && rank == 0) {
        if (lane == 0) {
            Issuer r;
            r.run<P, FP8>(c, sh, ring, tmem);
            if (!r.ok) sh->failed = 1;
        }
    } else if (run && warp == kWatchWarp && rank == 0) {
        Watcher r;
        r.turn = turn;
        if constexpr (P == kGrads) {
            if (a.job[0].M > 0) r.run<kDx, false>(a.job[0], c, g, sh, ring.stages, lane);
            if (a.job[1].M > 0) r.run<kDw, false>(a.job[1], c, g, sh, ring.stages, lane);
            if (a.job[2].M > 0) r.run<kDw, false>(a.job[2], c, g, sh, ring.stages, lane);
        } else {
            r.run<P, FP8>(a.job[0], c, g, sh, ring.stages, lane);
        }
        r.end(sh, lane);
        if (!r.ok) sh->failed = 1;
    } else if (run && warp >= 2 && warp < kWatchWarp) {
        Drain r;
        r.turn = turn;
        if (c.early) pdl_wait();
        uint8_t* turn_buf = turns + (warp - 2) * ffn_turn(P);
        if constexpr (P == kGrads) {
            if (a.job[0].M > 0) r.run<kDx, false>(a.job[0], c, g, sh, tmem, rank, warp, lane, turn_buf);
            if (a.job[1].M > 0) r.run<kDw, false>(a.job[1], c, g, sh, tmem, rank, warp, lane, turn_buf);
            if (a.job[2].M > 0) r.run<kDw, false>(a.job[2], c, g, sh, tmem, rank, warp, lane, turn_buf);
            if (lane == 0) bulk_wait<0>();
        } else {
            r.run<P, FP8>(a.job[0], c, g, sh, tmem, rank, warp, lane, turn_buf);
        }
        if (!r.ok) sh->failed = 1;
    } else if (P == kGrads && run && warp == kMendWarp) {
        if constexpr (P == kGrads) {
            Mender r;
            r.turn = turn;
            if (a.job[0].M > 0) r.run<kDx>(a.job[0], c, g, sh, ring, lane);
            if (a.job[1].M > 0) r.run<kDw>(a.job[1], c, g, sh, ring, lane);
            if (a.job[2].M > 0) r.run<kDw>(a.job[2], c, g, sh, ring, lane);
            if (!r.ok) sh->failed = 1;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (sh->failed) {  // time for the copies and instructions on their way to end before the block goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 20000000u) __nanosleep(1000);
        __syncthreads();
    }
    pair_arrive();
    pair_wait();  // neither block leaves while the other may still use its barriers or tensor memory
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

}  // namespace moe

// ---------------------------------------------------------------- host
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Row indexes and a tile's past them stay within 32 bits.
constexpr int64_t kMaxRows = (int64_t(1) << 31) - (1 << 24);

int check_sizes(int64_t rows, int E, int H, int I, const MoePlanOut* plan) {
    if (plan == nullptr || plan->cu_seqlens == nullptr || plan->tokens_per_expert == nullptr || plan->status == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRows || E < 1 || E > 1024 || H < 8 || H % 8 != 0 || H >= (1 << 20) || I < 8 ||
        I % 8 != 0 || I >= (1 << 20))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// A product's job: the weights and the rows (dw: the left and the right rows).
template <int P, bool FP8 = false>
int make_job(moe::Job* j, const void* weights, const void* row_data, int64_t rows, int E, int M, int N, int K,
             uint16_t* out) {
    constexpr int bytes = FP8 ? 1 : 2;
    j->M = M;
    j->N = N;
    j->K = K;
    j->out = out;
    // The thread that issues copies takes longer for a slice of many than the
    // products do (some 50 cycles each and 200 for the stage's wait): a block's
    // part of a slice is one copy where the extents allow it, with more
    // extents than the array has.  Gated: the M side's 16 channels of the gate
    // and of the up projection in turn, for M in whole 16s.  Transposed operands:
    // two runs of 64 elements, for whole 64s (a run that left its row would read
    // the next one's, and past the array's end at the last).
    const int run = 128 / bytes, box_k = run;
    const int64_t m = M, n = N, k = K, mk = m * k;
    int rc;
    if constexpr (P == moe::kGated) {
        j->m_whole = M % 16 == 0;
        if (j->m_whole)
            rc = moe_host::make_tensor_map(&j->map_m, weights, bytes,
                                           {{k, 1, box_k}, {16, k, 16}, {2, mk, 2}, {m / 16, 16 * k, 4}, {E, 2 * mk, 1}});
        else
            rc = moe_host::make_tensor_map(&j->map_m, weights, bytes, {{k, 1, box_k}, {m, k, 16}, {2, mk, 2}, {E, 2 * mk, 1}});
    } else if constexpr (P == moe::kDown) {
        rc = moe_host::make_tensor_map(&j->map_m, weights, 2, {{k, 1, run}, {m, k, moe::kHalf}, {E, mk, 1}});
    } else if constexpr (P == moe::kDw) {
        j->m_whole = M % 64 == 0;
        if (j->m_whole)
            rc = moe_host::make_tensor_map(&j->map_m, weights, 2, {{run, 1, run}, {rows, m, 64}, {m / run, run, 2}});
        else
            rc = moe_host::make_tensor_map(&j->map_m, weights, 2, {{m, 1, run}, {rows, m, 64}});
    } else {
        j->m_whole = M % 64 == 0;
        if (j->m_whole)
            rc = moe_host::make_tensor_map(&j->map_m, weights, 2, {{run, 1, run}, {k, m, 64}, {m / run, run, 2}, {E, mk, 1}});
        else
            rc = moe_host::make_tensor_map(&j->map_m, weights, 2, {{m, 1, run}, {k, m, 64}, {E, mk, 1}});
    }
    if (rc != MOE_OK) return rc;
    if constexpr (P == moe::kDw) {
        j->n_whole = N % 128 == 0;  // and a block's half of the last tile starts at a run
        if (j->n_whole)
            rc = moe_host::make_tensor_map(&j->map_n[0], row_data, 2, {{run, 1, run}, {rows, n, 64}, {n / run, run, 2}});
        else
            rc = moe_host::make_tensor_map(&j->map_n[0], row_data, 2, {{n, 1, run}, {rows, n, 64}});
        return rc != MOE_OK ? rc : moe_host::make_tensor_map(&j->map_out, out, 2, {{n, 1, run}, {m, n, 32}, {E, m * n, 1}});
    } else {
        for (int i = 0; i < 5 && rc == MOE_OK; ++i)
            rc = moe_host::make_tensor_map(&j->map_n[i], row_data, bytes, {{k, 1, box_k}, {rows, k, i == 0 ? 16 : 32 * i}});
        return rc;
    }
}

template <int P, bool FP8 = false>
int launch(moe::Launch<P>& a, cudaStream_t stream) {
    // as many stages of 32 KB as fit: six, five with dw
    constexpr size_t kSmem = 227 * 1024, kStage = 2 * moe::kHalf * moe::kSlice;
    const size_t fixed = 1024 + moe::kEpilogueWarps * moe::ffn_turn(P) + sizeof(moe::Shared) +
                         sizeof(int) * (4 * static_cast<size_t>(a.c.E) + 1);
    a.c.ring_bytes = static_cast<int>((kSmem - fixed) / kStage * kStage);
    static_assert(1024 + moe::kEpilogueWarps * 4096 + sizeof(moe::Shared) + sizeof(int) * 4097 + 5 * kStage <= kSmem, "shared memory");
    if (cudaFuncSetAttribute(moe::ffn_kernel<P, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem)) != cudaSuccess)
        return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(moe_host::num_sms() & ~1));
    cfg.blockDim = dim3(moe::ffn_threads(P));
    cfg.dynamicSmemBytes = fixed + a.c.ring_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = moe_host::pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, moe::ffn_kernel<P, FP8>, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe::Common common_of(const MoePlanOut* plan, int64_t rows, int E, int early) {
    moe::Common c = {};
    c.cu = plan->cu_seqlens;
    c.count = plan->tokens_per_expert;
    c.status = plan->status;
    c.rows = rows;
    c.E = E;
    c.early = early;
    c.timeout_ns = moe_host::timeout_ns();
    return c;
}

template <bool FP8>
int launch_gated(const void* x, const float* x_scale, const void* w_gate_up, const float* w_scale, int64_t rows, int E,
                 int H, int I, const MoePlanOut* plan, uint16_t* h, float* preact, cudaStream_t stream) {
    moe::Launch<moe::kGated> a = {};
    a.c = common_of(plan, rows, E, 0);
    a.c.a_scale = x_scale;
    a.c.b_scale = w_scale;
    a.c.preact_out = preact;
    const int rc = make_job<moe::kGated, FP8>(&a.job[0], w_gate_up, x, rows, E, I, 0, H, h);
    return rc != MOE_OK ? rc : launch<moe::kGated, FP8>(a, stream);
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
    const int rg = fp8 ? launch_gated<true>(x, x_scale, w_gate_up, w_scale, rows, E, H, I, plan, h, nullptr, stream)
                       : launch_gated<false>(x, nullptr, w_gate_up, nullptr, rows, E, H, I, plan, h, preact, stream);
    if (rg != MOE_OK) return rg;
    moe::Launch<moe::kDown> a = {};
    a.c = common_of(plan, rows, E, 1);
    const int rd = make_job<moe::kDown>(&a.job[0], w_down, h, rows, E, H, 0, I, y);
    return rd != MOE_OK ? rd : launch<moe::kDown>(a, stream);
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
    if (dx != nullptr || dw_gate_up != nullptr) {
        moe::Launch<moe::kDgate> a = {};
        a.c = common_of(plan, rows, E, 0);
        a.c.preact_in = preact;
        rc = make_job<moe::kDgate>(&a.job[0], w_down, dy, rows, E, I, 0, H, dgate_up);
        if (rc == MOE_OK) rc = launch<moe::kDgate>(a, stream);
        if (rc != MOE_OK) return rc;
    }
    if (dx == nullptr && dw_gate_up == nullptr && dw_down == nullptr) return MOE_OK;
    moe::Launch<moe::kGrads> a = {};
    a.c = common_of(plan, rows, E, dx != nullptr || dw_gate_up != nullptr);
    if (dx != nullptr) rc = make_job<moe::kDx>(&a.job[0], w_gate_up, dgate_up, rows, E, H, 0, 2 * I, dx);
    if (rc == MOE_OK && dw_gate_up != nullptr)
        rc = make_job<moe::kDw>(&a.job[1], dgate_up, x, rows, E, 2 * I, H, 0, dw_gate_up);
    if (rc == MOE_OK && dw_down != nullptr) rc = make_job<moe::kDw>(&a.job[2], dy, h, rows, E, H, I, 0, dw_down);
    return rc != MOE_OK ? rc : launch<moe::kGrads>(a, stream);
}
