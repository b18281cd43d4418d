// block_norm.cu -- the norms between two blocks, with the gate and the scaled
// residual, and their gradient (sm_103a).
//
// Forward, for a row x (a block's output) and r (the residual stream):
//   n = x * rp * wp,  rp = 1 / sqrt(mean(x^2) + eps)   the norm after the block,
//   s = a r + c n                                      gate c, residual scale a,
//   v = s * rs * w,   rs = 1 / sqrt(mean(s^2) + eps)   the norm before the next one,
// v in bf16 and, on request, in 8 bits.  One pass: x, r and the gate come in
// once, s stays in registers (fp32) between the row's two sums and its maximum.
//
// Backward, with sh = s rs, xh = x rp, t = dy w:
//   d  = rs (t - sh mean(t sh)) + ds      the gradient of s,
//   dr = a d,  dc = d n,
//   dx = rp (e - xh mean(e xh)),  e = d c wp,
//   dw = sum over rows of dy sh,  dwp = sum over rows of d c xh.
// A row has two sums, the second over what the first one gives; with a gate for
// each token both the gate's gradient and mean(e xh) come from sum(d n).  The
// weights' sums stay in registers over a block's rows (a thread keeps its
// columns); partial rows are joined in block order by a second launch.
//
// Memory bound: every element is read once and written once.  Forms as in
// norm.cu: a warp a row (H <= 512), a block a row (past 8192 columns the gradient
// spills registers: right, but not tuned), and for many rows a ring of rows in
// shared memory (which rows, and both sides' figures: forward_ring_rows,
// backward_ring_rows).
// Measured (GB300, copy rate 6.80 TB/s): forward with a gate a token and the 8-bit
// output at 8192 x 7168, 95 us, 5.6 TB/s (a block a row: 124 us); with fp32 sums and a gate
// an element at 16384 x 4096, 144 us, 6.5 TB/s; backward at 16384 x 4096 with
// fp32 sums 200 us, 6.0 TB/s (a block a row: 234), at 8192 x 7168 with a gate an element
// 158 us, 5.9 TB/s (282).
#include "norm_parts.cuh"

namespace moe {

enum Gate { kNoGate = 0, kTokenGate = 1, kFullGate = 2 };

// A row's root or gate.  Volatile: not before the wait for the launch ahead, which may write it.  (Cached: a
// line has 32 rows' values.)
__device__ __forceinline__ float row_value(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

struct BlockNormArgs {
    const uint16_t* x;
    const void* residual;
    const void* gate;  // float32[N] or bf16[N][H]
    const void* post_weight;
    const void* weight;
    int post_f32, weight_f32;
    int N, H;
    float alpha, eps;
    float down, mean;  // of the squares' sums (square_scale)
    uint16_t* y;
    void* residual_out;
    float* post_rstd;
    float* rstd;
    uint8_t* q;
    float* q_scale;
};

// 1 / sqrt(mean(v^2) + eps) of a row held in registers.
template <int VPT, bool WARP>
__device__ __forceinline__ float row_root(const float (&v)[VPT][8], int lane, int lanes, int nvec, const BlockNormArgs& a,
                                          float* buf) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (lane + i * lanes < nvec)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = v[i][j] * a.down;
                ss = fmaf(t, t, ss);
            }
    ss = row_reduce<WARP, false>(ss, buf);
    float root = rsqrtf(fmaf(ss, a.mean, a.eps));  // within 2^-22
    if (!(fmaf(ss, a.mean, a.eps) >= kLeastEps)) {
        // Squares may have lost digits below the normal numbers, or vanished, and
        // eps does not cover them: no value is above 2^-42, all are summed again,
        // scaled.  (The row's threads hold the same sum and take the same way.)
        constexpr float kUp = 0x1p90f;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (lane + i * lanes < nvec)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = v[i][j] * kUp;
                    ss = fmaf(t, t, ss);
                }
        ss = row_reduce<WARP, false>(ss, buf) * (a.down * a.down);
        root = kUp * rsqrtf(fmaf(ss, a.mean, a.eps * kUp * kUp));
    }
    return root;
}

template <int VPT, bool WARP, typename R, int GATE>
__global__ void __launch_bounds__(WARP ? 128 : 256 * VPT) block_norm_kernel(const BlockNormArgs a) {
    __shared__ float buf[32];
    pdl_wait();
    pdl_trigger();
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int lanes = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.N) return;
    const int nvec = a.H / 8;
    const int64_t at = row * a.H;
    const R* residual = static_cast<const R*>(a.residual) + at;
    const uint16_t* gate = static_cast<const uint16_t*>(a.gate) + at;

    // Everything the row needs is asked for before the first sum is waited for;
    // the widest rows (VPT 4) have no registers for that.
    constexpr bool kEarly = VPT <= 2;
    float s[VPT][8], r[kEarly ? VPT : 1][8], g[kEarly && GATE == kFullGate ? VPT : 1][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * lanes;
        if (c < nvec) {
            load8(a.x + at, c, s[i]);
            if constexpr (kEarly) load8_written(residual, c, r[i]);
            if constexpr (kEarly && GATE == kFullGate) load8(gate, c, g[i]);
        }
    }
    const float token_gate = GATE == kTokenGate ? row_value(static_cast<const float*>(a.gate) + row) : 1.f;
    const float post = row_root<VPT, WARP>(s, lane, lanes, nvec, a, buf);
    if (lane == 0) a.post_rstd[row] = post;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * lanes;
        if (c < nvec) {
            constexpr int kOwn = kEarly ? 1 : 0;  // the place of chunk i: its own, or the only one
            if constexpr (!kEarly) load8_written(residual, c, r[0]);
            if constexpr (!kEarly && GATE == kFullGate) load8(gate, c, g[0]);
            float w[8];
            load_weight8(a.post_weight, a.post_f32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float n = s[i][j] * post * w[j];
                if constexpr (GATE == kTokenGate) n *= token_gate;
                if constexpr (GATE == kFullGate) n *= g[i * kOwn][j];
                s[i][j] = fmaf(a.alpha, r[i * kOwn][j], n);
            }
            store8(static_cast<R*>(a.residual_out) + at, c, s[i]);
        }
    }
    const float rstd = row_root<VPT, WARP>(s, lane, lanes, nvec, a, buf);
    if (lane == 0) a.rstd[row] = rstd;

    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * lanes;
        if (c < nvec) {
            float w[8];
            load_weight8(a.weight, a.weight_f32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[i][j] = s[i][j] * rstd * w[j];
                amax = fmaxf(amax, fabsf(s[i][j]));
            }
            store8(a.y + at, c, s[i]);
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

// ---------------------------------------------------------------- ring
// A warp has 256 columns of the block's rows, a lane eight of them.  The warp's lanes copy its columns of
// the next rows into shared memory (cp.async, 16 bytes a lane, side by side) while the block works on a
// row; only the warp reads them, so that a slot needs no barrier of the block.  (Eight bytes a thread, the
// columns it needs itself, go through L1, which the ring leaves little of: 8192 x 7168 in 110 us, so in 97.)
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_columns(uint16_t* to, const uint16_t* row, int first, int H) {
    const int h = first + 8 * (threadIdx.x & 31);
    if (h < H) copy16(to + h, row + h);
}
__device__ __forceinline__ void copy_columns(float* to, const float* row, int first, int H) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int h = first + 128 * i + 4 * (threadIdx.x & 31);
        if (h < H) copy16(to + h, row + h);
    }
}

// The lane's eight columns: one run, or where there are fp32 rows (SPLIT) two runs of four, 128 columns apart, so
// that the lanes' 16 bytes of an fp32 row are side by side.
template <bool SPLIT>
struct Columns {
    int at;         // the first run's
    bool in0, in1;  // the runs are inside the row
    __device__ __forceinline__ explicit Columns(int H) {
        at = threadIdx.x / 32 * 256 + (SPLIT ? 4 : 8) * (threadIdx.x & 31);
        in0 = at < H;
        in1 = (SPLIT ? at + 128 : at) < H;
    }
    // Of a row in the ring, whose places behind its end hold zeros.
    template <typename T>
    __device__ __forceinline__ void read(const T* row, float (&f)[8]) const {
        if constexpr (SPLIT) {
            float v[4];
            load4(row + at, v);
            f[0] = v[0], f[1] = v[1], f[2] = v[2], f[3] = v[3];
            load4(row + at + 128, v);
            f[4] = v[0], f[5] = v[1], f[6] = v[2], f[7] = v[3];
        } else {
            unpack8(*reinterpret_cast<const uint4*>(row + at), f);
        }
    }
    template <typename T>
    __device__ __forceinline__ void write(T* row, const float (&f)[8]) const {
        if constexpr (SPLIT) {
            const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
            if (in0) store4(row + at, a);
            if (in1) store4(row + at + 128, b);
        } else {
            if (in0) store8(row, at / 8, f);
        }
    }
    __device__ __forceinline__ void write(uint8_t* row, const Quantum& q, const float (&f)[8]) const {
        const uint32_t a = q.round4(f), b = q.round4(f + 4);
        if constexpr (SPLIT) {
            if (in0) *reinterpret_cast<uint32_t*>(row + at) = a;
            if (in1) *reinterpret_cast<uint32_t*>(row + at + 128) = b;
        } else {
            if (in0) *reinterpret_cast<uint2*>(row + at) = make_uint2(a, b);
        }
    }
    __device__ __forceinline__ void weights(const void* w, int f32, float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int h = at + j + (SPLIT && j >= 4 ? 124 : 0);
            f[j] = !(j < 4 ? in0 : in1) ? 0.f
                   : f32                ? static_cast<const float*>(w)[h]
                                        : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(w)[h]) << 16);
        }
    }
};

// Until at most slots - 1 of the thread's groups of copies are under way, and the warp's have landed.
__device__ __forceinline__ void ring_wait(int slots) {
    if (slots == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
    __syncwarp();
}

// Zeros in the places behind the rows' end (and everywhere else), before the first copies: the columns of
// rows of `bytes` a slot.
__device__ __forceinline__ void ring_clear(uint8_t* smem, uint32_t bytes) {
    for (uint32_t v = 16 * threadIdx.x; v < bytes; v += 16 * blockDim.x)
        *reinterpret_cast<uint4*>(smem + v) = make_uint4(0, 0, 0, 0);
    __syncthreads();
}

// Two elements at a time: the arithmetic of a pair is one instruction, and these kernels' rows of
// two-byte elements are bound by instructions and barriers before memory.
struct Pair {
    uint64_t v;
};
__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 parts(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
    return f;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
    return p;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return p;
}
__device__ __forceinline__ float sum_of(Pair p) {
    const float2 f = parts(p);
    return f.x + f.y;
}
__device__ __forceinline__ Pair both(float f) { return pair(f, f); }
__device__ __forceinline__ void split(const float (&f)[8], Pair (&p)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = pair(f[2 * j], f[2 * j + 1]);
}
__device__ __forceinline__ void join(const Pair (&p)[4], float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = parts(p[j]);
        f[2 * j] = v.x, f[2 * j + 1] = v.y;
    }
}
template <bool SPLIT, typename T>
__device__ __forceinline__ void read(const Columns<SPLIT>& c, const T* row, Pair (&p)[4]) {
    float f[8];
    c.read(row, f);
    split(f, p);
}

// The block's sum of one value and maximum of another, with one barrier.  buf: two of 32 floats, and as
// block_reduce's one of two sets.
__device__ __forceinline__ float2 sum_and_max(float v, float m, float (*buf)[32]) {
    auto fold = [&] {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v += __shfl_xor_sync(FULL_MASK, v, o);
            m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
        }
    };
    fold();
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[0][threadIdx.x >> 5] = v, buf[1][threadIdx.x >> 5] = m;
    __syncthreads();
    const bool there = lane < static_cast<int>(blockDim.x >> 5);
    v = there ? buf[0][lane] : 0.f;
    m = there ? buf[1][lane] : 0.f;
    fold();
    return make_float2(v, m);
}

// The least product s * w * 2^32 of a row whose largest |v| is taken from it: it is a normal number with room to
// spare.  Where the largest is below, or infinite (a weight of 2^96, or both large), the row's threads, which hold the
// same value, take the maximum of |v| itself; of ordinary rows only those of zeros.  (The way out costs 8192 x 7168
// 2.5%, 94.8 us against 92.5: other registers and order, not the test.  The power of two by the block's weights, or a
// loop of its own for large ones, cost 6%.)
constexpr float kLeastProduct = 0x1p-58f;

// A row's place holds its columns rounded up to whole warps'.
__host__ __device__ __forceinline__ int ring_columns(int H) { return (H + 255) / 256 * 256; }

// R: the residual's element type.  slots: 2 or 3.
template <typename R, int GATE>
__global__ void __launch_bounds__(kRingThreads) block_norm_ring_kernel(const BlockNormArgs a, const int slots) {
    extern __shared__ __align__(16) uint8_t smem[];  // [slots][x row, gate row, residual row]
    __shared__ float buf[2][3][32];
    pdl_wait();
    pdl_trigger();
    const int H = a.H, W = ring_columns(H), first = threadIdx.x / 32 * 256;
    const Columns<sizeof(R) == 4> mine(H);
    constexpr int kNarrow = GATE == kFullGate ? 2 : 1;  // rows of two bytes an element
    const uint32_t slot_bytes = static_cast<uint32_t>(W) * (2 * kNarrow + sizeof(R));
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.N / gridDim.x;
    const int64_t end = (static_cast<int64_t>(blockIdx.x) + 1) * a.N / gridDim.x;
    auto fetch = [&](int64_t row, int slot) {
        __syncwarp();  // all lanes have read what was there
        if (row < end) {
            uint16_t* x = reinterpret_cast<uint16_t*>(smem + slot * slot_bytes);
            copy_columns(x, a.x + row * H, first, H);
            if constexpr (GATE == kFullGate) copy_columns(x + W, static_cast<const uint16_t*>(a.gate) + row * H, first, H);
            copy_columns(reinterpret_cast<R*>(x + kNarrow * W), static_cast<const R*>(a.residual) + row * H, first, H);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Pair wp[4], w[4];
    float f[8];
    mine.weights(a.post_weight, a.post_f32, f);
    split(f, wp);
    mine.weights(a.weight, a.weight_f32, f);
    split(f, w);
    if (H != W) ring_clear(smem, slots * slot_bytes);
    for (int j = 0; j < slots - 1; ++j) fetch(begin + j, j);
    const Pair down = both(a.down), alpha = both(a.alpha);
    float next_gate = GATE == kTokenGate && begin < end ? row_value(static_cast<const float*>(a.gate) + begin) : 1.f;
    int slot = 0;  // the row's
    for (int64_t row = begin; row < end; ++row) {
        fetch(row + slots - 1, slot == 0 ? slots - 1 : slot - 1);
        const Pair token_gate = both(next_gate);
        if (GATE == kTokenGate && row + 1 < end) next_gate = row_value(static_cast<const float*>(a.gate) + row + 1);
        ring_wait(slots);
        const uint16_t* x = reinterpret_cast<const uint16_t*>(smem + slot * slot_bytes);
        slot = slot + 1 == slots ? 0 : slot + 1;
        const int64_t at = row * H;
        Pair s[4], sum = both(0.f);
        read(mine, x, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Pair t = s[j] * down;
            sum = fma(t, t, sum);
        }
        const float post_root = rsqrtf(fmaf(block_reduce<false>(sum_of(sum), buf[row & 1][0]), a.mean, a.eps));  // within 2^-22
        if (threadIdx.x == 0) a.post_rstd[row] = post_root;
        const Pair post = both(post_root);
        Pair q[4], g[4];
        read(mine, reinterpret_cast<const R*>(x + kNarrow * W), q);
        if constexpr (GATE == kFullGate) read(mine, x + W, g);
        // The row's largest |v| comes with its sum, as that of s * w * 2^32 (kLeastProduct).
        float amax = 0.f;
        sum = both(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Pair n = s[j] * post * wp[j];
            if constexpr (GATE == kTokenGate) n = n * token_gate;
            if constexpr (GATE == kFullGate) n = n * g[j];
            s[j] = fma(alpha, q[j], n);
            const Pair t = s[j] * down;
            sum = fma(t, t, sum);
            const float2 u = parts(s[j] * (w[j] * both(0x1p32f)));
            amax = fmaxf(amax, fmaxf(fabsf(u.x), fabsf(u.y)));
        }
        join(s, f);
        mine.write(static_cast<R*>(a.residual_out) + at, f);
        const float2 joined = sum_and_max(sum_of(sum), amax, buf[row & 1] + 1);
        const float root = rsqrtf(fmaf(joined.x, a.mean, a.eps));
        if (threadIdx.x == 0) a.rstd[row] = root;
        const Pair rstd = both(root);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = s[j] * rstd * w[j];
        join(s, f);
        mine.write(a.y + at, f);
        if (a.q == nullptr) continue;
        amax = joined.y * 0x1p-32f * root;
        if (!(joined.y >= kLeastProduct && joined.y < INFINITY)) {
            amax = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
            amax = row_reduce<false, true>(amax, buf[row & 1][0]);
        }
        const Quantum quantum = quantum_of(amax);
        if (threadIdx.x == 0) a.q_scale[row] = quantum.scale;
        mine.write(a.q + at, quantum, f);
    }
}

// ---------------------------------------------------------------- backward
struct BlockNormBackwardArgs {
    const uint16_t* dy;
    const uint16_t* x;
    const void* s;
    const void* ds;  // may be null
    const void* gate;
    const void* post_weight;
    const void* weight;
    int post_f32, weight_f32;
    const float* post_rstd;
    const float* rstd;
    int N, H;
    float alpha;
    uint16_t* dx;
    void* dres;
    void* dgate;  // float32[N] or bf16[N][H]
    float* partial;  // [gridDim.x][2][H]: dweight's, dpost_weight's
};

template <int VPT, bool WARP, typename S, int GATE>
__global__ void __launch_bounds__(WARP ? 128 : 256 * VPT) block_norm_backward_kernel(const BlockNormBackwardArgs a) {
    extern __shared__ float sh[];  // WARP: [warps][2][H] for the block's sums
    __shared__ float buf[32];
    pdl_wait();
    pdl_trigger();
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int lanes = WARP ? 32 : blockDim.x;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    const int per_step = WARP ? warps : 1;
    const int nvec = a.H / 8;
    const float over_h = 1.f / static_cast<float>(a.H);

    float acc[VPT][8], post_acc[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = post_acc[i][j] = 0.f;
    // rows of a block are consecutive: its partial sums have a fixed order
    const int64_t steps = (static_cast<int64_t>(a.N) + per_step - 1) / per_step;
    const int64_t begin = blockIdx.x * steps / gridDim.x, end = (blockIdx.x + 1) * steps / gridDim.x;
    for (int64_t step = begin; step < end; ++step) {
        const int64_t row = WARP ? step * per_step + warp : step;
        if (row >= a.N) break;
        const int64_t at = row * a.H;
        const float rstd = row_value(a.rstd + row), post = row_value(a.post_rstd + row);
        const float token_gate = GATE == kTokenGate ? row_value(static_cast<const float*>(a.gate) + row) : 1.f;
        const uint16_t* gate = static_cast<const uint16_t*>(a.gate) + at;
        float hat[VPT][8], t[VPT][8], d[VPT][8], xh[VPT][8];  // all is asked for before the row's first sum
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] = 0.f;
            if (c < nvec) {
                load8(a.dy + at, c, t[i]);
                load8(static_cast<const S*>(a.s) + at, c, hat[i]);
                load8(a.x + at, c, xh[i]);
                if (a.ds != nullptr) load8(static_cast<const S*>(a.ds) + at, c, d[i]);
            }
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) {
                float w[8];
                load_weight8(a.weight, a.weight_f32, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    hat[i][j] *= rstd;
                    xh[i][j] *= post;
                    acc[i][j] = fmaf(t[i][j], hat[i][j], acc[i][j]);
                    t[i][j] *= w[j];
                    dot = fmaf(t[i][j], hat[i][j], dot);
                }
            }
        }
        const float mean = row_reduce<WARP, false>(dot, buf) * over_h;
        dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) {
                float w[8], g[8], o[8];
                load_weight8(a.post_weight, a.post_f32, c, w);
                if constexpr (GATE == kFullGate) load8(gate, c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d[i][j] += rstd * (t[i][j] - hat[i][j] * mean);
                    o[j] = a.alpha * d[i][j];
                }
                store8(static_cast<S*>(a.dres) + at, c, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = xh[i][j] * w[j];
                    if constexpr (GATE == kFullGate) {
                        o[j] = d[i][j] * n;
                        d[i][j] *= g[j];
                        dot = fmaf(d[i][j], n, dot);
                    } else {
                        dot = fmaf(d[i][j], n, dot);
                        d[i][j] *= token_gate;
                    }
                    post_acc[i][j] = fmaf(d[i][j], xh[i][j], post_acc[i][j]);
                    d[i][j] *= w[j];
                }
                if constexpr (GATE == kFullGate) store8(static_cast<uint16_t*>(a.dgate) + at, c, o);
            }
        }
        dot = row_reduce<WARP, false>(dot, buf);
        if constexpr (GATE == kTokenGate) {
            if (lane == 0) static_cast<float*>(a.dgate)[row] = dot;
            dot *= token_gate;
        }
        const float post_mean = dot * over_h;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = post * (d[i][j] - xh[i][j] * post_mean);
                store8(a.dx + at, c, d[i]);
            }
        }
    }
    float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
    if constexpr (WARP) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) {
                store8(sh + (2 * warp) * a.H, c, acc[i]);
                store8(sh + (2 * warp + 1) * a.H, c, post_acc[i]);
            }
        }
        __syncthreads();
        for (int h = threadIdx.x; h < 2 * a.H; h += blockDim.x) {
            float v = 0.f;
            for (int k = 0; k < warps; ++k) v += sh[2 * k * a.H + h];
            out[h] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * lanes;
            if (c < nvec) {
                store8(out, c, acc[i]);
                store8(out + a.H, c, post_acc[i]);
            }
        }
    }
}

// A thread reads its columns' values from the ring anew in each of the row's three parts: in
// registers there is only room for what has no other place (the weights' sums and d).
template <typename S, int GATE, bool DS>
__global__ void __launch_bounds__(kRingThreads) block_norm_backward_ring_kernel(const BlockNormBackwardArgs a,
                                                                               const int slots) {
    extern __shared__ __align__(16) uint8_t smem[];  // [slots][dy row, x row, gate row, s row, ds row]
    __shared__ float buf[2][2][32];
    pdl_wait();
    pdl_trigger();
    const int H = a.H, W = ring_columns(H), first = threadIdx.x / 32 * 256;
    const Columns<sizeof(S) == 4> mine(H);
    constexpr int kNarrow = GATE == kFullGate ? 3 : 2;  // rows of two bytes an element
    const uint32_t slot_bytes = static_cast<uint32_t>(W) * (2 * kNarrow + (DS ? 2 : 1) * sizeof(S));
    const float over_h = 1.f / static_cast<float>(H);
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.N / gridDim.x;
    const int64_t end = (static_cast<int64_t>(blockIdx.x) + 1) * a.N / gridDim.x;
    auto fetch = [&](int64_t row, int slot) {
        __syncwarp();  // all lanes have read what was there
        if (row < end) {
            uint16_t* dy = reinterpret_cast<uint16_t*>(smem + slot * slot_bytes);
            S* s = reinterpret_cast<S*>(dy + kNarrow * W);
            copy_columns(dy, a.dy + row * H, first, H);
            copy_columns(s, static_cast<const S*>(a.s) + row * H, first, H);
            copy_columns(dy + W, a.x + row * H, first, H);
            if constexpr (DS) copy_columns(s + W, static_cast<const S*>(a.ds) + row * H, first, H);
            if constexpr (GATE == kFullGate)
                copy_columns(dy + 2 * W, static_cast<const uint16_t*>(a.gate) + row * H, first, H);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Pair w[4], wp[4], acc[4], post_acc[4];
    float o[8];
    mine.weights(a.weight, a.weight_f32, o);
    split(o, w);
    mine.weights(a.post_weight, a.post_f32, o);
    split(o, wp);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = post_acc[j] = both(0.f);
    if (H != W) ring_clear(smem, slots * slot_bytes);
    for (int j = 0; j < slots - 1; ++j) fetch(begin + j, j);
    int slot = 0;  // the row's
    float next_rstd = 0.f, next_post = 0.f, next_gate = 1.f;
    auto scalars = [&](int64_t row) {
        if (row >= end) return;
        next_rstd = row_value(a.rstd + row);
        next_post = row_value(a.post_rstd + row);
        if constexpr (GATE == kTokenGate) next_gate = row_value(static_cast<const float*>(a.gate) + row);
    };
    scalars(begin);
    for (int64_t row = begin; row < end; ++row) {
        fetch(row + slots - 1, slot == 0 ? slots - 1 : slot - 1);
        const Pair rstd = both(next_rstd), post = both(next_post);
        const float token_gate = next_gate;
        scalars(row + 1);
        ring_wait(slots);
        const uint16_t* dy = reinterpret_cast<const uint16_t*>(smem + slot * slot_bytes);
        slot = slot + 1 == slots ? 0 : slot + 1;
        const S* s = reinterpret_cast<const S*>(dy + kNarrow * W);
        const int64_t at = row * H;
        float(*sums)[32] = buf[row & 1];
        Pair t[4], v[4], d[4], sum = both(0.f);
        read(mine, dy, t);
        read(mine, s, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = v[j] * rstd;
            acc[j] = fma(t[j], v[j], acc[j]);
            sum = fma(t[j] * w[j], v[j], sum);
        }
        const Pair mean = both(-block_reduce<false>(sum_of(sum), sums[0]) * over_h);
        read(mine, dy, t);
        read(mine, s, v);
        if constexpr (DS) read(mine, s + W, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Pair u = fma(v[j] * rstd, mean, t[j] * w[j]);
            if constexpr (DS) d[j] = fma(rstd, u, d[j]);
            else d[j] = rstd * u;
            v[j] = both(a.alpha) * d[j];
        }
        join(v, o);
        mine.write(static_cast<S*>(a.dres) + at, o);
        read(mine, dy + W, v);
        if constexpr (GATE == kFullGate) read(mine, dy + 2 * W, t);
        sum = both(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = v[j] * post;
            const Pair n = v[j] * wp[j];
            sum = fma(d[j], GATE == kFullGate ? n * t[j] : n, sum);
            if constexpr (GATE == kFullGate) {
                const Pair c = t[j];
                t[j] = d[j] * n;
                d[j] = d[j] * c;
            }
            if constexpr (GATE == kTokenGate) d[j] = d[j] * both(token_gate);
            post_acc[j] = fma(d[j], v[j], post_acc[j]);
            d[j] = d[j] * wp[j];
        }
        if constexpr (GATE == kFullGate) {
            join(t, o);
            mine.write(static_cast<uint16_t*>(a.dgate) + at, o);
        }
        float dot = block_reduce<false>(sum_of(sum), sums[1]);
        if constexpr (GATE == kTokenGate) {
            if (threadIdx.x == 0) static_cast<float*>(a.dgate)[row] = dot;
            dot *= token_gate;
        }
        const Pair post_mean = both(-dot * over_h);
        read(mine, dy + W, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = post * fma(v[j] * post, post_mean, d[j]);
        join(d, o);
        mine.write(a.dx + at, o);
    }
    float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * H;
    join(acc, o);
    mine.write(out, o);
    join(post_acc, o);
    mine.write(out + H, o);
}

// The weights' gradients from the blocks' partials: 32 columns a block; each
// of its 32 warps adds every 32nd partial, and the warps' sums are joined in order.
__global__ void __launch_bounds__(1024) block_norm_weights_kernel(const float* partial, int blocks, int H, float* dweight,
                                                                  float* dpost) {
    __shared__ float sh[32][33];
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x * 32 + threadIdx.x, g = threadIdx.y;
    float v = 0.f;
    if (h < 2 * H) {
#pragma unroll 4
        for (int b = g; b < blocks; b += 32) v += partial[static_cast<int64_t>(b) * 2 * H + h];
    }
    sh[g][threadIdx.x] = v;
    __syncthreads();
    v = warp_sum(sh[threadIdx.x][g]);  // warp g joins column g
    const int c = blockIdx.x * 32 + g;
    if (threadIdx.x == 0 && c < 2 * H) (c < H ? dweight[c] : dpost[c - H]) = v;
}

}  // namespace moe

// ---------------------------------------------------------------- host
namespace {

using namespace moe_host;

template <int VPT, bool WARP, typename R>
int launch_gate(const moe::BlockNormArgs& a, int gate, dim3 grid, dim3 block, cudaStream_t stream) {
    switch (gate) {
        case moe::kNoGate: return launch(moe::block_norm_kernel<VPT, WARP, R, moe::kNoGate>, grid, block, 0, stream, a);
        case moe::kTokenGate: return launch(moe::block_norm_kernel<VPT, WARP, R, moe::kTokenGate>, grid, block, 0, stream, a);
        default: return launch(moe::block_norm_kernel<VPT, WARP, R, moe::kFullGate>, grid, block, 0, stream, a);
    }
}

template <int VPT, bool WARP>
int launch_forward(const moe::BlockNormArgs& a, bool f32, int gate, dim3 grid, dim3 block, cudaStream_t stream) {
    return f32 ? launch_gate<VPT, WARP, float>(a, gate, grid, block, stream)
               : launch_gate<VPT, WARP, uint16_t>(a, gate, grid, block, stream);
}

template <int VPT, bool WARP, typename S>
int launch_backward_gate(const moe::BlockNormBackwardArgs& a, int gate, dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream) {
    switch (gate) {
        case moe::kNoGate:
            return launch(moe::block_norm_backward_kernel<VPT, WARP, S, moe::kNoGate>, grid, block, smem, stream, a);
        case moe::kTokenGate:
            return launch(moe::block_norm_backward_kernel<VPT, WARP, S, moe::kTokenGate>, grid, block, smem, stream, a);
        default: return launch(moe::block_norm_backward_kernel<VPT, WARP, S, moe::kFullGate>, grid, block, smem, stream, a);
    }
}

template <int VPT, bool WARP>
int launch_backward(const moe::BlockNormBackwardArgs& a, bool f32, int gate, dim3 grid, dim3 block, size_t smem,
                    cudaStream_t stream) {
    return f32 ? launch_backward_gate<VPT, WARP, float>(a, gate, grid, block, smem, stream)
               : launch_backward_gate<VPT, WARP, uint16_t>(a, gate, grid, block, smem, stream);
}

// The ring form of these kernels, with `bytes` a column of a row in a slot.  A row has two sums one after the
// other, in which a block only waits: so an SM has as many blocks as its threads (64 registers each) allow,
// but not more than ask for `ahead` bytes at a time.  More than that in flight, by more blocks or more slots,
// costs up to a sixth again, and less does too.  Share of the copy rate with half of `ahead`, this, and twice this:
// forward, bf16 sums and a gate a token, 32000 x 2048 69, 87, 87%; 16384 x 4096 68, 85, 85%; fp32 sums and a gate an
// element, 16384 x 4096 95, 95, 86%; gradient with bf16 sums 16384 x 4096 51, 90, 90%, with a gate an element
// 8192 x 7168 90, 90, 78%; with fp32 sums 32000 x 2048 71, 95, 95%, 16384 x 4096 94, 88, 88%.  A third slot is for
// blocks that are alone on their SM and small.
struct BlockRing {
    int slots = 0, threads = 0, blocks = 0;  // slots = 0: there is none
    size_t smem = 0;
};
constexpr int kMostBlocks = 8;  // of an SM
constexpr size_t kForwardAhead = 36 * 1024, kBackwardAhead = 96 * 1024;
BlockRing block_ring_for(int H, int bytes, size_t ahead, int sms) {
    constexpr size_t kSmem = 220 * 1024;
    const size_t slot = static_cast<size_t>(moe::ring_columns(H)) * bytes;
    BlockRing r;
    if (H <= 512 || H > 8 * moe::kRingThreads || 2 * slot > kSmem) return r;
    const int threads = moe::ring_columns(H) / 8;
    int per_sm = moe::kRingThreads / threads;
    if (per_sm > kMostBlocks) per_sm = kMostBlocks;
    while (per_sm > 1 && (per_sm * slot > ahead || 2 * per_sm * slot > kSmem)) --per_sm;
    r.slots = per_sm == 1 && 3 * slot <= kSmem && (slot <= kForwardAhead || threads <= moe::kRingThreads / 2) ? 3 : 2;
    r.threads = threads;
    r.blocks = sms * per_sm;
    r.smem = r.slots * slot;
    return r;
}

template <typename Kernel, typename Args>
int launch_block_ring(Kernel kernel, const BlockRing& r, const Args& a, cudaStream_t stream) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) != cudaSuccess)
        return MOE_ERR_CUDA;
    return launch(kernel, dim3(static_cast<unsigned>(r.blocks)), dim3(static_cast<unsigned>(r.threads)), r.smem, stream, a,
                  r.slots);
}

template <typename R>
int launch_forward_ring(const BlockRing& r, const moe::BlockNormArgs& a, int gate, cudaStream_t stream) {
    switch (gate) {
        case moe::kNoGate: return launch_block_ring(moe::block_norm_ring_kernel<R, moe::kNoGate>, r, a, stream);
        case moe::kTokenGate: return launch_block_ring(moe::block_norm_ring_kernel<R, moe::kTokenGate>, r, a, stream);
        default: return launch_block_ring(moe::block_norm_ring_kernel<R, moe::kFullGate>, r, a, stream);
    }
}

template <typename S, bool DS>
int launch_backward_ring(const BlockRing& r, const moe::BlockNormBackwardArgs& a, int gate, cudaStream_t stream) {
    switch (gate) {
        case moe::kNoGate: return launch_block_ring(moe::block_norm_backward_ring_kernel<S, moe::kNoGate, DS>, r, a, stream);
        case moe::kTokenGate:
            return launch_block_ring(moe::block_norm_backward_ring_kernel<S, moe::kTokenGate, DS>, r, a, stream);
        default: return launch_block_ring(moe::block_norm_backward_ring_kernel<S, moe::kFullGate, DS>, r, a, stream);
    }
}

bool ring_taken(const BlockRing& r, int N, int rows) { return r.slots > 0 && N / rows >= r.blocks; }

// Rows a block from which the forward kernel takes the ring; 0: never.  Wide rows after a few (block a row, ring, us:
// 7168 bf16 620 rows 10.6, 10.9, 2600 rows 39.9, 32.5, with a gate an element 63.1, 35.6; 4096 bf16 1300 rows 10.9, 11.6,
// 5000 rows 37.8, 32.8; 4096 fp32 with a gate an element 14.8, 15.6 and 53.7, 47.0), bf16 rows of 1024 to 2048 columns
// later (1024: 10000 rows 15.3, 17.8, 40000 rows 58.6, 56.4; 2048: 5000 rows 15.9, 18.4, 32000 rows 95.5, 88.9), fp32 rows
// up to there and narrower ones never (2048 fp32 32000 rows 137, 145; 640 bf16 65536 rows 70, 86).  Where the rule is off:
// bf16 rows of 1024 to 2048 columns with a gate an element (32000 x 2048 110, 118) and fp32 rows of 2056 to 4096 without
// one (20000 x 2056 83, 107; 16384 x 4096 123, 134).
int forward_ring_rows(int H, bool f32) { return H > 2048 ? 4 : H >= 1024 && !f32 ? 16 : 0; }

// The gradient's ring, by the bytes of a column of its rows, and the rows a block from which it is taken.
BlockRing backward_ring(int H, int bytes, int sms) { return block_ring_for(H, bytes, kBackwardAhead, sms); }
// Wide rows take it as soon as every block has one (block a row, ring, us: 7168 bf16 160 rows 15.4, 12.6, 8192 rows
// 219, 121; 2048 bf16 1300 rows 16.9, 14.3, 32000 rows 207, 132); narrow ones after four (1000 bf16 1300 rows 11.9, 13.7,
// 5000 rows 22.5, 21.5, 65536 rows 211, 140, fp32 with a gate a token 24.3, 25.8 and 230, 188; 640 bf16 65536 rows 177,
// 118).
int backward_ring_rows(int H) { return H >= 2048 ? 1 : 4; }

// Blocks of the backward kernel's other forms: four an SM, no more than there are rows.
int backward_blocks(int N, int H, int sms) {
    const int64_t units = H <= 512 ? (static_cast<int64_t>(N) + 3) / 4 : N;
    const int64_t cap = static_cast<int64_t>(sms) * 4;
    return static_cast<int>(units < cap ? units : cap);
}

// For the most blocks of any call with these rows or fewer: a caller's workspace for its largest batch serves all.
size_t backward_workspace(int N, int H, int sms) {
    const int rows = backward_ring_rows(H);
    int blocks = 1;
    for (int bytes = 6; bytes <= 14; bytes += 2) {  // dy, x; sums of 2 or 4 bytes, twice with ds; a gate an element
        const BlockRing ring = backward_ring(H, bytes, sms);
        const bool taken = ring_taken(ring, N, rows);
        const int others = backward_blocks(taken ? ring.blocks * rows - 1 : N, H, sms);
        if (others > blocks) blocks = others;
        if (taken && ring.blocks > blocks) blocks = ring.blocks;
    }
    return static_cast<size_t>(blocks) * 2 * H * sizeof(float);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A gate is float32[N] or bf16[N][H]; 0: there is none, -1: not a gate.
int gate_of(const void* gate, int gate_dtype) {
    if (gate == nullptr) return moe::kNoGate;
    if (gate_dtype == MOE_DTYPE_F32) return aligned4(gate) ? moe::kTokenGate : -1;
    if (gate_dtype == MOE_DTYPE_BF16) return aligned16(gate) ? moe::kFullGate : -1;
    return -1;
}

}  // namespace

extern "C" MOE_API int moe_block_norm(const uint16_t* x, const void* residual, int residual_dtype, const void* gate,
                                      int gate_dtype, const void* post_weight, int post_weight_dtype, const void* weight,
                                      int weight_dtype, int N, int H, float residual_scale, float eps, uint16_t* y,
                                      void* residual_out, float* post_rstd, float* rstd, uint8_t* q, float* q_scale,
                                      cudaStream_t stream) {
    if (N < 0 || H < 8 || H % 8 != 0 || !(eps >= 0.f) || std::isinf(eps) || !std::isfinite(residual_scale))
        return MOE_ERR_INVALID_ARG;
    if (!float_type(post_weight_dtype) || !float_type(weight_dtype) || !float_type(residual_dtype))
        return MOE_ERR_INVALID_ARG;
    const int kind = gate_of(gate, gate_dtype);
    if (kind < 0) return MOE_ERR_INVALID_ARG;
    if (N > 0 && (x == nullptr || residual == nullptr || post_weight == nullptr || weight == nullptr || y == nullptr ||
                  residual_out == nullptr || post_rstd == nullptr || rstd == nullptr || (q == nullptr) != (q_scale == nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(post_weight) || !aligned16(weight) || !aligned16(y) ||
        !aligned16(residual_out) || !aligned4(post_rstd) || !aligned4(rstd) || !aligned4(q_scale) ||
        (reinterpret_cast<uintptr_t>(q) & 7u) != 0)
        return MOE_ERR_INVALID_ARG;
    if (H > kMaxH) return MOE_ERR_UNSUPPORTED;
    if (N == 0) return MOE_OK;
    float down, mean;
    square_scale(H, &down, &mean);
    const bool f32 = residual_dtype == MOE_DTYPE_F32;
    const moe::BlockNormArgs a = {x, residual, gate, post_weight, weight, post_weight_dtype == MOE_DTYPE_F32,
                                  weight_dtype == MOE_DTYPE_F32, N, H, residual_scale, eps, down, mean, y,
                                  residual_out, post_rstd, rstd, q, q_scale};
    const int rows = forward_ring_rows(H, f32);
    // (the ring has no second sum for squares that vanish: only with an eps that covers them)
    if (eps >= moe::kLeastEps && rows > 0) {
        const BlockRing ring = block_ring_for(H, 2 + (f32 ? 4 : 2) + (kind == moe::kFullGate ? 2 : 0), kForwardAhead,
                                              num_sms());
        if (ring_taken(ring, N, rows))
            return f32 ? launch_forward_ring<float>(ring, a, kind, stream) : launch_forward_ring<uint16_t>(ring, a, kind, stream);
    }
    if (H <= 512) {
        const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(N) + 3) / 4)), block(128);
        return H <= 256 ? launch_forward<1, true>(a, f32, kind, grid, block, stream)
                        : launch_forward<2, true>(a, f32, kind, grid, block, stream);
    }
    const dim3 grid(static_cast<unsigned>(N)), block(static_cast<unsigned>(norm_threads(H)));
    switch (norm_vpt(H)) {
        case 1: return launch_forward<1, false>(a, f32, kind, grid, block, stream);
        case 2: return launch_forward<2, false>(a, f32, kind, grid, block, stream);
        default: return launch_forward<4, false>(a, f32, kind, grid, block, stream);
    }
}

extern "C" MOE_API size_t moe_block_norm_backward_workspace_size(int N, int H) {
    if (N < 0 || H < 8 || H % 8 != 0 || H > kMaxH) return 0;
    return backward_workspace(N, H, num_sms());
}

extern "C" MOE_API int moe_block_norm_backward(const uint16_t* dy, const uint16_t* x, const void* s, int s_dtype,
                                               const void* ds, const void* gate, int gate_dtype, const void* post_weight,
                                               int post_weight_dtype, const void* weight, int weight_dtype,
                                               const float* post_rstd, const float* rstd, int N, int H,
                                               float residual_scale, uint16_t* dx, void* dres, void* dgate,
                                               float* dpost_weight, float* dweight, void* workspace,
                                               size_t workspace_bytes, cudaStream_t stream) {
    if (N < 0 || H < 8 || H % 8 != 0 || !std::isfinite(residual_scale)) return MOE_ERR_INVALID_ARG;
    if (!float_type(post_weight_dtype) || !float_type(weight_dtype) || !float_type(s_dtype)) return MOE_ERR_INVALID_ARG;
    const int kind = gate_of(gate, gate_dtype);
    if (kind < 0 || (gate == nullptr && dgate != nullptr)) return MOE_ERR_INVALID_ARG;
    if (dweight == nullptr || dpost_weight == nullptr) return MOE_ERR_INVALID_ARG;
    if (N > 0 && (dy == nullptr || x == nullptr || s == nullptr || post_weight == nullptr || weight == nullptr ||
                  post_rstd == nullptr || rstd == nullptr || dx == nullptr || dres == nullptr || workspace == nullptr ||
                  (gate != nullptr) != (dgate != nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(s) || !aligned16(ds) || !aligned16(post_weight) ||
        !aligned16(weight) || !aligned16(dx) || !aligned16(dres) || !aligned16(workspace) || !aligned4(post_rstd) ||
        !aligned4(rstd) || !aligned4(dweight) || !aligned4(dpost_weight) ||
        !(kind == moe::kFullGate ? aligned16(dgate) : aligned4(dgate)))
        return MOE_ERR_INVALID_ARG;
    if (H > kMaxH) return MOE_ERR_UNSUPPORTED;
    if (N == 0) {
        if (cudaMemsetAsync(dweight, 0, sizeof(float) * H, stream) != cudaSuccess ||
            cudaMemsetAsync(dpost_weight, 0, sizeof(float) * H, stream) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    const int sms = num_sms();
    if (workspace_bytes < backward_workspace(N, H, sms)) return MOE_ERR_CAPACITY;
    const bool f32 = s_dtype == MOE_DTYPE_F32;
    const BlockRing ring =
        backward_ring(H, 4 + (ds != nullptr ? 2 : 1) * (f32 ? 4 : 2) + (kind == moe::kFullGate ? 2 : 0), sms);
    const bool taken = ring_taken(ring, N, backward_ring_rows(H));
    const int blocks = taken ? ring.blocks : backward_blocks(N, H, sms);
    float* partial = static_cast<float*>(workspace);
    const moe::BlockNormBackwardArgs a = {dy, x, s, ds, gate, post_weight, weight, post_weight_dtype == MOE_DTYPE_F32,
                                          weight_dtype == MOE_DTYPE_F32, post_rstd, rstd, N, H, residual_scale, dx, dres,
                                          dgate, partial};
    const dim3 grid(static_cast<unsigned>(blocks));
    int rc;
    if (taken) {
        if (ds != nullptr)
            rc = f32 ? launch_backward_ring<float, true>(ring, a, kind, stream)
                     : launch_backward_ring<uint16_t, true>(ring, a, kind, stream);
        else
            rc = f32 ? launch_backward_ring<float, false>(ring, a, kind, stream)
                     : launch_backward_ring<uint16_t, false>(ring, a, kind, stream);
    } else if (H <= 512) {
        const dim3 block(128);
        const size_t smem = 8 * sizeof(float) * H;
        rc = H <= 256 ? launch_backward<1, true>(a, f32, kind, grid, block, smem, stream)
                      : launch_backward<2, true>(a, f32, kind, grid, block, smem, stream);
    } else {
        const dim3 block(static_cast<unsigned>(norm_threads(H)));
        switch (norm_vpt(H)) {
            case 1: rc = launch_backward<1, false>(a, f32, kind, grid, block, 0, stream); break;
            case 2: rc = launch_backward<2, false>(a, f32, kind, grid, block, 0, stream); break;
            default: rc = launch_backward<4, false>(a, f32, kind, grid, block, 0, stream); break;
        }
    }
    if (rc != MOE_OK) return rc;
    return launch(moe::block_norm_weights_kernel, dim3(static_cast<unsigned>((2 * H + 31) / 32)), dim3(32, 32), 0, stream,
                  static_cast<const float*>(partial), blocks, H, dweight, dpost_weight);
}
