// anvil_head.cu -- softmax cross entropy of a head z = x W^T over a large vocabulary, without the logits
// in memory.
//
//   forward   lse = log sum_j e^z_j, loss = lse - z_t
//   gradient  d_j = g (e^(z_j - lse) - [j = t]),  dx = d W,  dW = d^T x
//
// Forward: the pair kernel (anvil_linear.cuh), whose epilogue takes each tile's logits out of tensor
// memory once and leaves, per row and 64 columns, their maximum and the sum of their exponentials
// over it (8 bytes for 64 logits), and the target's logit where it is among them.  A second kernel joins a
// row's pairs.  8192 x 50304 x 768 bf16: 380 us, 1.67 PFLOP/s, the tensor pipe active 78% of the time; from
// k = 256 down the epilogue bounds it (3205 x 98816 x 152: 155 us, about 4600 cycles a tile).
//
// Gradient: the logits again, a piece of the vocabulary at a time.  The epilogue turns them into d, 16
// bits, the operand of both products that follow: dW's rows of the piece are complete, dx is added up
// in fp32 over the pieces.  So the workspace is bounded whatever the vocabulary, and the flops are the
// three products' 6 rows vocab k.  8192 x 50304 x 768 bf16: 1080 to 1130 us, 1.7 PFLOP/s.
//
// Exponentials in powers of two, one fused operation and one of the hardware's powers each (struct Base), over
// the largest logit itself: lse = m + log S, so that a logit that stands alone is its row's lse to the bit.
#include <cuda_runtime.h>
#include <stdint.h>

#include "anvil_linear.cuh"

namespace anvil {

namespace {

constexpr float LOG2E = 1.44269504f;

// 2^v, of results below 2^-126 0 (a relative error of 2^-22; the subnormal results would cost as much again).
__device__ __forceinline__ float exp2_of(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ uint64_t exp2_of(uint64_t v) {
    float lo, hi;
    f2_split(v, &lo, &hi);
    return f2_make(exp2_of(lo), exp2_of(hi));
}

// e^(z - m) = 2^(z by - base) undo, by = log2(e).  base = m by is rounded; what that drops is the same in every
// z's power, 2^rest, and undo = 2^-rest takes it out again.  From |m| = 2^29 on rest passes 32 and would soon
// overflow, but fp32 values are 64 apart there: by = 1 takes any other z than m to nothing as well, and base is m.
struct Base {
    float by, base;
    __device__ __forceinline__ explicit Base(float m) {
        by = fabsf(m) >= 0x1p29f ? 1.f : LOG2E;
        base = __fmul_rn(m, by);
    }
    __device__ __forceinline__ float rest(float m) const { return by == 1.f ? 0.f : __fmaf_rn(m, by, -base); }
};

__device__ __forceinline__ long long target_of(const void* targets, int wide, long long row) {
    return wide ? static_cast<const long long*>(targets)[row] : static_cast<const int*>(targets)[row];
}
// Column of the target relative to `first` as an int; -1 where it is before it or beyond any column.
__device__ __forceinline__ int relative_target(const PairHeadParams& p, long long row) {
    const long long t = target_of(p.targets, p.target64, row) - p.first;
    return t >= 0 && t < p.cols ? static_cast<int>(t) : -1;
}

struct StatsPair {
    using Params = PairHeadParams;
    static constexpr bool MULTI = false, OWN = true, RANK_B = false, ONE_CHAIN = false;
    static constexpr int CHAIN = 0;
    struct Row {
        long long row;
        int target;
    };
    static __device__ __forceinline__ Row load(const Params& p, const Unit& t, int r) {
        const long long row = static_cast<long long>(t.tr) * PAIR_ROWS + r;
        return {row, row < p.rows && p.hit ? relative_target(p, row) : -1};
    }
    template <typename T, int W>
    static __device__ __forceinline__ void tile(const Params& p, EpiState& x, uint32_t tacc, uint32_t tempty, const Unit& t,
                                                int, const Row& row) {
        static_assert(EPI_COLS == HEAD_STATS_COLS, "one pair of statistics per group and row");
        const int col0 = t.tc * BN + x.grp * EPI_COLS;
        const uint32_t ta = tacc + x.grp * EPI_COLS;
        const int live = p.cols - col0;  // columns of this group that exist
        float most = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int h = 0; h < EPI_COLS; h += 32) {
            float v[32];
            tmem_ld_32x32b_x32(ta + h, v);
            if (live < h + 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (h + i >= live) v[i] = -INFINITY;
            }
            float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int i = 4; i < 32; ++i) m[i & 3] = fmaxf(m[i & 3], v[i]);
            const float now = fmaxf(most, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
            const float ref = now == -INFINITY ? 0.f : now;
            const Base e(ref);
            const uint64_t by = f2_make(e.by, e.by), less = f2_make(-e.base, -e.base);
            uint64_t s[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 32; i += 2) s[i / 2 & 1] = f2_add(s[i / 2 & 1], exp2_of(f2_fma(f2_make(v[i], v[i + 1]), by, less)));
            float s0, s1;
            f2_split(f2_add(s[0], s[1]), &s0, &s1);
            // (of an empty sum the factor does not count, but for being a number)
            sum = fmaf(s0 + s1, exp2_of(-e.rest(ref)), sum * exp2_of(fminf((most - now) * LOG2E, 0.f)));
            most = now;
        }
        const int at = row.target - col0;
        const bool mine = row.target >= 0 && at >= 0 && at < EPI_COLS;
        if (__any_sync(0xffffffffu, mine)) {  // one warp and tile in twenty at a vocabulary of 50,000
            float hit = 0.f;
#pragma unroll 1
            for (int c = 0; c < EPI_COLS; c += 16) {
                float v[16];
                tmem_ld_16(ta + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (at == c + i) hit = v[i];
            }
            if (mine) p.hit[row.row] = hit;
        }
        release_acc(x, tempty);
        if (row.row < p.rows) p.stats[static_cast<long long>(t.tc * EPI_GROUPS + x.grp) * p.rows + row.row] = make_float2(most == -INFINITY ? 0.f : most, sum);
    }
};

// The same of logits that are added up in registers, 1024 terms by the tensor cores at a time, for longer
// contractions.  The tensor cores' sums are cut off, which takes about 1.5e-8 of a logit at every 16 terms: at k = 65536
// one chain left lse 2.6e-4 too low (logits of deviation 2), this 3.5e-6.  512 terms would halve that, and cost 10% of the time
// at 2048 x 32000 x 4096 where 1024 cost 4% (about 297, 309 and 323 us); up to 1024 one chain is taken, in the kernel above,
// since the 64 sums of a thread hold its epilogue up (8192 x 50304 x 256: 173 us above, 187 here).
struct StatsChains {
    using Params = PairHeadParams;
    static constexpr bool MULTI = false, OWN = true, RANK_B = false, ONE_CHAIN = false;
    static constexpr int CHAIN = HEAD_CHAIN_KB;
    using Row = StatsPair::Row;
    static __device__ __forceinline__ Row load(const Params& p, const Unit& t, int r) { return StatsPair::load(p, t, r); }
    // v: this thread's row of the columns from col0 on
    template <typename T, int W>
    static __device__ __forceinline__ void tile(const Params& p, EpiState&, float (&v)[EPI_COLS], int, int col0, const Row& row) {
        static_assert(EPI_COLS == HEAD_STATS_COLS, "one pair of statistics per group and row");
        const int at = row.target - col0;
        const bool mine = row.target >= 0 && at >= 0 && at < EPI_COLS;
        if (__any_sync(0xffffffffu, mine)) {  // one warp and tile in twenty at a vocabulary of 50,000
            float hit = 0.f;
#pragma unroll
            for (int i = 0; i < EPI_COLS; ++i)
                if (at == i) hit = v[i];
            if (mine) p.hit[row.row] = hit;
        }
        const int live = p.cols - col0;  // columns that exist
        if (live < EPI_COLS) {
#pragma unroll
            for (int i = 0; i < EPI_COLS; ++i)
                if (i >= live) v[i] = -INFINITY;
        }
        float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int i = 4; i < EPI_COLS; ++i) m[i & 3] = fmaxf(m[i & 3], v[i]);
        const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));  // (NaN where all are, and so is the sum)
        const float ref = most == -INFINITY ? 0.f : most;
        const Base e(ref);
        const uint64_t by = f2_make(e.by, e.by), less = f2_make(-e.base, -e.base);
        uint64_t s[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < EPI_COLS; i += 2) s[i / 2 & 3] = f2_add(s[i / 2 & 3], exp2_of(f2_fma(f2_make(v[i], v[i + 1]), by, less)));
        float s0, s1;
        f2_split(f2_add(f2_add(s[0], s[1]), f2_add(s[2], s[3])), &s0, &s1);
        if (row.row < p.rows)
            p.stats[static_cast<long long>(col0 / EPI_COLS) * p.rows + row.row] = make_float2(ref, (s0 + s1) * exp2_of(-e.rest(ref)));
    }
};

struct DlogitsPair {
    using Params = PairHeadParams;
    static constexpr bool MULTI = false, OWN = true, RANK_B = false, ONE_CHAIN = false;
    static constexpr int CHAIN = 0;
    struct Row {
        float by, less;   // e^(z - lse) = 2^(z by + less) / one
        float one, g;     // d = (2^(z by + less) - [j = target] one) g
        uint32_t counts;  // all ones, or 0 where the gradient is 0 whatever the logits are
        int target;
    };
    static __device__ __forceinline__ Row load(const Params& p, const Unit& t, int r) {
        const long long row = static_cast<long long>(t.tr) * PAIR_ROWS + r;
        Row x = {0.f, 0.f, 1.f, 0.f, 0u, -1};
        if (row < p.rows && target_of(p.targets, p.target64, row) >= 0) {
            const float lse = p.lse[row];
            if (lse != -INFINITY) {  // (no token of that row can be: its gradient is 0)
                const Base e(lse);
                const float rest = e.rest(lse), g = p.grad[row] * *p.scale;
                x.by = e.by;
                x.less = -e.base;
                x.one = exp2_of(rest);
                x.g = g * exp2_of(-rest);
                x.counts = g == 0.f ? 0u : 0xffffffffu;
                x.target = relative_target(p, row);
            }
        }
        return x;
    }
    // Sixteen logits from column c of the box on; hot: the target's number among them, if it is.
    template <typename T, int W>
    static __device__ __forceinline__ void sixteen(const EpiState& x, float (&v)[16], int c, int hot, const Row& row) {
        const uint64_t by = f2_make(row.by, row.by), less = f2_make(row.less, row.less), g = f2_make(row.g, row.g);
#pragma unroll
        for (int i = 0; i < 16; i += 2) f2_split(exp2_of(f2_fma(f2_make(v[i], v[i + 1]), by, less)), &v[i], &v[i + 1]);
        if (row.target >= 0 && hot >= 0 && hot < 16) {  // one warp and sixteen columns in a hundred, of 50,000
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (hot == i) v[i] -= row.one;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint64_t d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = f2_mul(f2_make(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]), g);
            uint4 w = Elem<T>::pack_pairs(d);
            w.x &= row.counts;
            w.y &= row.counts;
            w.z &= row.counts;
            w.w &= row.counts;
            sts128(Staging<W>::addr(x.box, x.r, c / 8 + j), w);
        }
    }
    // (the buffer's rows go on in eights: no box ends inside 16 bytes)
    template <int W>
    static __device__ __forceinline__ void send(const Params& p, const EpiState& x, int row0, int col) {
        send_box<uint16_t, W, true>(x, &p.tm_out, 1, p.epi.out, p.epi.ldout, row0, col, p.rows, (p.cols + 7) & ~7);
    }
    template <typename T, int W>
    static __device__ __forceinline__ void tile(const Params& p, EpiState& x, uint32_t tacc, uint32_t tempty, const Unit& t,
                                                int row0, const Row& row) {
        constexpr int COLS = W / 2, N = EPI_COLS / COLS;
        const int col0 = t.tc * BN + x.grp * EPI_COLS;
        const uint32_t ta = tacc + x.grp * EPI_COLS;
        const int at = row.target - col0;
#pragma unroll 1
        for (int b = 0; b < N; ++b) {
            box_free(x);
#pragma unroll 1
            for (int c = 0; c < COLS; c += 16) {
                float v[16];
                tmem_ld_16(ta + b * COLS + c, v);
                sixteen<T, W>(x, v, c, at - (b * COLS + c), row);
            }
            if (b == N - 1) release_acc(x, tempty);
            send<W>(p, x, row0, col0 + b * COLS);
        }
    }
};

// The same of the logits that StatsChains takes (from one chain the probabilities would not fit lse: at k = 65536
// they would be 0.1% off).
struct DlogitsChains {
    using Params = PairHeadParams;
    static constexpr bool MULTI = false, OWN = true, RANK_B = false, ONE_CHAIN = false;
    static constexpr int CHAIN = HEAD_CHAIN_KB;
    using Row = DlogitsPair::Row;
    static __device__ __forceinline__ Row load(const Params& p, const Unit& t, int r) { return DlogitsPair::load(p, t, r); }
    template <typename T, int W>
    static __device__ __forceinline__ void tile(const Params& p, EpiState& x, float (&v)[EPI_COLS], int row0, int col0, const Row& row) {
        constexpr int COLS = W / 2;
        const int at = row.target - col0;
#pragma unroll
        for (int c = 0; c < EPI_COLS; c += 16) {
            if (c % COLS == 0) box_free(x);
            float u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = v[c + i];
            DlogitsPair::sixteen<T, W>(x, u, c % COLS, at - c, row);
            if (c % COLS == COLS - 16) DlogitsPair::send<W>(p, x, row0, col0 + c - c % COLS);
        }
    }
};

// Two sums over different logits as one.  (A part with a sum of 0 has no logit above -inf; a NaN goes
// through the sums.)
__device__ __forceinline__ void join(float& ref, float& sum, float ref2, float sum2) {
    const float now = sum2 == 0.f ? ref : sum == 0.f ? ref2 : fmaxf(ref, ref2);
    sum = (sum == 0.f ? 0.f : sum * exp2_of((ref - now) * LOG2E)) + (sum2 == 0.f ? 0.f : sum2 * exp2_of((ref2 - now) * LOG2E));
    ref = now;
}

// Eight values of every lane combined over the warp; lane l gets number l / 4's.
template <class Op>
__device__ __forceinline__ float gather8(float (&v)[8], int lane, Op op) {
#pragma unroll
    for (int half = 4, bit = 16; half > 0; half /= 2, bit /= 2) {
        const bool upper = lane & bit;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, bit));
        }
    }
    v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// Few rows: a thread has one column's logits of eight rows, a warp 32 columns, a block 128.
struct HeadRows {
    using Params = RowHeadParams;
    static constexpr bool GATED = false, HEAD = true;
    static constexpr int BLOCKS = 3;
    static __device__ __forceinline__ void finish(const Params& p, const float (&v)[8], int col, bool live, int row, int rows, float2* to) {
        // over the warp's columns: each exchange halves the rows that a lane goes on with, until lane l has
        // row l / 4's, from where every lane gets all eight maxima
        const int lane = threadIdx.x & 31;
        float m[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = live ? v[i] : -INFINITY;
        const float most = gather8(m, lane, [](float a, float b) { return fmaxf(a, b); });
        const float mine = most == -INFINITY ? 0.f : most;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Base e(__shfl_sync(0xffffffffu, mine, 4 * i));
            s[i] = live ? exp2_of(fmaf(v[i], e.by, -e.base)) : 0.f;
        }
        const float sum = gather8(s, lane, [](float a, float b) { return a + b; });
        if (lane % 4 == 0) to[lane / 4] = make_float2(mine, sum * exp2_of(-Base(mine).rest(mine)));
        if (p.hit) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (live && i < rows && target_of(p.targets, p.target64, row + i) == col) p.hit[row + i] = v[i];
        }
    }
    static __device__ __forceinline__ void end(const Params& p, int block, int row, float2 a, float2 b, float2 c, float2 d) {
        join(a.x, a.y, b.x, b.y);
        join(c.x, c.y, d.x, d.y);
        join(a.x, a.y, c.x, c.y);
        p.stats[static_cast<long long>(block) * p.nb + row] = a;
    }
};

// One or two rows and a small weight: read once, by warps that take four of its rows at a time and keep
// each token's running statistics; no tensor cores, no tiles to fill.  A lane takes every 32nd 16-byte chunk,
// twelve of them on their way, the tokens wait in shared memory as fp32.  One row, us with the join, against the
// row kernel: 5000 x 768 6.5/8.3, 8000 x 4096 15.4/17.8; 20000 x 768 10.8/9.4, 50304 x 768 18.3/17.4, 32000 x
// 4096 47.2/44.6.  (Three blocks an SM, with fewer registers each, were slower.)
template <typename T, int R>
__global__ void __launch_bounds__(32 * HEAD_TOKEN_WARPS, 2) head_token_kernel(const TokenHeadParams p) {
    constexpr int G = HEAD_TOKEN_GROUP, E = Elem<T>::VEC;
    extern __shared__ __align__(16) float token_values[];  // [R][chunks * E]
    float* const xs = token_values;
    __shared__ float2 shares[HEAD_TOKEN_WARPS][R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (p.k + E - 1) / E, whole = p.k / E;
    const long long step = static_cast<long long>(gridDim.x) * HEAD_TOKEN_WARPS * G;
    pdl_allow_next();
    pdl_wait_previous();
    for (int i = threadIdx.x; i < R * chunks * E; i += 32 * HEAD_TOKEN_WARPS) {
        const int r = i / (chunks * E), c = i - r * chunks * E;
        xs[i] = c < p.k && r < p.rows ? Elem<T>::load(static_cast<const T*>(p.x)[r * p.ldx + c]) : 0.f;
    }
    __syncthreads();
    float ref = 0.f, sum = 0.f;  // lane r's: token r
    const long long target = p.hit && lane < p.rows ? target_of(p.targets, p.target64, lane) : -1;
    for (long long row0 = (static_cast<long long>(blockIdx.x) * HEAD_TOKEN_WARPS + warp) * G; row0 < p.cols; row0 += step) {
        const T* w[G];
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = static_cast<const T*>(p.w) + min(row0 + g, static_cast<long long>(p.cols) - 1) * p.ldw;
        uint64_t acc[G][R];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[g][r] = 0;
        constexpr int U = 3;  // chunks of a lane on their way at a time
        for (int c0 = lane; c0 - lane < chunks; c0 += 32 * U) {
            uint4 in[U][G];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    in[u][g] = c0 + 32 * u < whole ? ldg_stream(w[g] + (c0 + 32 * u) * E) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + 32 * u;
                if (c == whole && whole < chunks) {  // the row's last values
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        float f[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) f[e] = c * E + e < p.k ? Elem<T>::load(w[g][c * E + e]) : 0.f;
                        in[u][g] = Elem<T>::pack(f);
                    }
                }
                if (c >= chunks) break;
                uint64_t wv[G][E / 2];
#pragma unroll
                for (int g = 0; g < G; ++g) Elem<T>::unpack_pairs(in[u][g], wv[g]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4* q = reinterpret_cast<const float4*>(xs + (r * chunks + c) * E);
                    const float4 a = q[0], b = q[1];
                    const uint64_t xv[4] = {f2_make(a.x, a.y), f2_make(a.z, a.w), f2_make(b.x, b.y), f2_make(b.z, b.w)};
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) acc[g][r] = f2_fma(wv[g][e], xv[e], acc[g][r]);
                }
            }
        }
        float z[G];  // of token `lane`
#pragma unroll
        for (int g = 0; g < G; ++g) {
            z[g] = -INFINITY;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float lo, hi;
                f2_split(acc[g][r], &lo, &hi);
                float v = lo + hi;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == r) z[g] = v;
            }
        }
        if (lane < R) {
            float most = -INFINITY;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (row0 + g >= p.cols) z[g] = -INFINITY;
                else if (row0 + g == target) p.hit[lane] = z[g];
                most = fmaxf(most, z[g]);
            }
            const float m = most == -INFINITY ? 0.f : most;
            const Base e(m);
            float s = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (row0 + g < p.cols) s += exp2_of(fmaf(z[g], e.by, -e.base));
            join(ref, sum, m, s * exp2_of(-e.rest(m)));
        }
    }
    if (lane < R) shares[warp][lane] = make_float2(ref, sum);
    __syncthreads();
    if (threadIdx.x < p.rows) {
        ref = shares[0][threadIdx.x].x;
        sum = shares[0][threadIdx.x].y;
        for (int k = 1; k < HEAD_TOKEN_WARPS; ++k) join(ref, sum, shares[k][threadIdx.x].x, shares[k][threadIdx.x].y);
        p.stats[static_cast<long long>(blockIdx.x) * p.rows + threadIdx.x] = make_float2(ref, sum);
    }
}

// A row's statistics joined, in a fixed order.  A block takes four rows, neighbours in the statistics (32
// bytes), and 64 shares of the parts: 8 in a warp, joined by shuffles, and 8 warps.
constexpr int HJ_ROWS = 4, HJ_THREADS = 256, HJ_SHARES = HJ_THREADS / HJ_ROWS, HJ_UNROLL = 4;
__global__ void __launch_bounds__(HJ_THREADS) head_join_kernel(const HeadJoinParams p) {
    __shared__ float2 share[HJ_THREADS / 32][HJ_ROWS];
    const int x = threadIdx.x % HJ_ROWS, y = threadIdx.x / HJ_ROWS;
    const long long row = static_cast<long long>(blockIdx.x) * HJ_ROWS + x;
    pdl_allow_next();
    pdl_wait_previous();
    float ref = 0.f, sum = 0.f;
    if (row < p.rows) {
        for (int i0 = y; i0 < p.parts; i0 += HJ_SHARES * HJ_UNROLL) {
            float2 s[HJ_UNROLL];
#pragma unroll
            for (int k = 0; k < HJ_UNROLL; ++k) {
                const int i = i0 + k * HJ_SHARES;
                s[k] = i < p.parts ? __ldcs(&p.stats[static_cast<long long>(i) * p.rows + row]) : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < HJ_UNROLL; ++k) join(ref, sum, s[k].x, s[k].y);
        }
    }
#pragma unroll
    for (int o = HJ_ROWS; o < 32; o *= 2) {
        const float r2 = __shfl_xor_sync(0xffffffffu, ref, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        join(ref, sum, r2, s2);
    }
    if ((threadIdx.x & 31) < HJ_ROWS) share[threadIdx.x >> 5][x] = make_float2(ref, sum);
    __syncthreads();
    if (threadIdx.x >= HJ_ROWS || row >= p.rows) return;
    for (int k = 1; k < HJ_THREADS / 32; ++k) join(ref, sum, share[k][x].x, share[k][x].y);
    const float lse = sum == 0.f ? -INFINITY : ref + logf(sum);
    if (p.lse) p.lse[row] = lse;
    if (p.loss) {
        const long long t = target_of(p.targets, p.target64, row);
        p.loss[row] = t < 0 ? 0.f : t >= p.vocab ? NAN : lse == -INFINITY ? INFINITY : lse - p.hit[row];
    }
}

// d is taken over the largest |g|, which the products' results are multiplied by: a mean's g, the same
// in every row, would be rounded to 16 bits the same way in each, 2^-9 of every gradient, and in fp16
// most of d would be below the smallest value (2^-25; there 2^13 more).
__global__ void __launch_bounds__(1024) head_scale_kernel(const HeadScaleParams p) {
    __shared__ uint32_t warps[32];
    pdl_allow_next();
    pdl_wait_previous();
    uint32_t most = 0;
#pragma unroll 8
    for (long long i = threadIdx.x; i < p.rows; i += 1024) {
        const uint32_t g = __float_as_uint(p.grad[i]) & 0x7fffffffu;
        // (an infinity or a NaN makes its row what it is over any scale)
        most = max(most, target_of(p.targets, p.target64, i) >= 0 && g < 0x7f800000u ? g : 0u);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = most;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    most = __reduce_max_sync(0xffffffffu, warps[threadIdx.x]);
    if (threadIdx.x == 0) {
        float unit = __uint_as_float(most);
        // 0, and beyond 2^100 either way: as they are
        unit = unit >= 7.8886090522101181e-31f && unit <= 1.2676506002282294e30f ? (p.f16 ? unit * 0x1p-13f : unit) : 1.f;
        p.scale[0] = __fdiv_rn(1.f, unit);
        p.scale[1] = unit;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) head_round_kernel(const HeadRoundParams p) {
    pdl_allow_next();
    pdl_wait_previous();
    const float scale = *p.scale;
    const int chunks = (p.cols + 7) / 8;
    const long long ld = chunks * 8ll;  // (src's rows go on in eights)
    const bool vec = p.cols % 8 == 0 && p.ldd % 8 == 0 && !(reinterpret_cast<uintptr_t>(p.dst) & 15);
    for (Walk at(chunks, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256); at.row < p.rows; at.next(chunks)) {
        const long long row = at.row;
        const int c = at.chunk * 8;
        float v[8];
        Elem<float>::unpack(ldg_stream(p.src + row * ld + c), v);
        Elem<float>::unpack(ldg_stream(p.src + row * ld + c + 4), v + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
        T* to = static_cast<T*>(p.dst) + row * p.ldd + c;
        if (vec) {
            *reinterpret_cast<uint4*>(to) = Elem<T>::pack(v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < p.cols) to[e] = Elem<T>::store(v[e]);
        }
    }
}

constexpr int STATS_BOX = 0, DLOGITS_BOX = 64;  // seven and six stages: the products bound both kernels

}  // namespace

cudaError_t head_prepare() {
    cudaError_t e;
#define ANVIL_SMEM(kernel, bytes) \
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))) return e
#define ANVIL_HEAD(T)                                                                                    \
    ANVIL_SMEM((pair_gemm_kernel<T, STATS_BOX, StatsPair>), Staging<STATS_BOX>::SMEM);                   \
    ANVIL_SMEM((pair_chain_kernel<T, STATS_BOX, StatsChains>), Staging<STATS_BOX>::SMEM);                \
    ANVIL_SMEM((pair_gemm_kernel<T, DLOGITS_BOX, DlogitsPair>), Staging<DLOGITS_BOX>::SMEM);             \
    ANVIL_SMEM((pair_chain_kernel<T, DLOGITS_BOX, DlogitsChains>), Staging<DLOGITS_BOX>::SMEM);          \
    ANVIL_SMEM((head_token_kernel<T, 1>), 4 * (HEAD_TOKEN_VALUES + 8));                                  \
    ANVIL_SMEM((head_token_kernel<T, 2>), 4 * (HEAD_TOKEN_VALUES + 16));                                 \
    ANVIL_SMEM((row_gemm_kernel<T, 16, HeadRows>), RowShape<16>::smem(RowShape<16>::STAGES));            \
    ANVIL_SMEM((row_gemm_kernel<T, 32, HeadRows>), RowShape<32>::smem(RowShape<32>::STAGES))
    ANVIL_HEAD(__nv_bfloat16);
    ANVIL_HEAD(__half);
#undef ANVIL_HEAD
#undef ANVIL_SMEM
    return cudaSuccess;
}

namespace {
template <typename T, int W, typename ONE, typename CHAINS>
cudaError_t run_logits(const PairHeadParams& p, int sm_count, cudaStream_t s) {
    return p.k > HEAD_CHAIN_KB * GEMM_BK ? run_pair<T, W, CHAINS>(p, sm_count, s) : run_pair<T, W, ONE>(p, sm_count, s);
}
}  // namespace

cudaError_t launch_head_stats(const PairHeadParams& p, int sm_count, cudaStream_t s) {
    return p.f16 ? run_logits<__half, STATS_BOX, StatsPair, StatsChains>(p, sm_count, s)
                 : run_logits<__nv_bfloat16, STATS_BOX, StatsPair, StatsChains>(p, sm_count, s);
}

cudaError_t launch_head_dlogits(const PairHeadParams& p, int sm_count, cudaStream_t s) {
    return p.f16 ? run_logits<__half, DLOGITS_BOX, DlogitsPair, DlogitsChains>(p, sm_count, s)
                 : run_logits<__nv_bfloat16, DLOGITS_BOX, DlogitsPair, DlogitsChains>(p, sm_count, s);
}

namespace {
template <typename T>
cudaError_t pick_rows(const RowHeadParams& p, int bn, int sm_count, cudaStream_t s) {
    return bn == 16 ? run_row<T, 16, HeadRows>(p, sm_count, s) : run_row<T, 32, HeadRows>(p, sm_count, s);
}
}  // namespace

cudaError_t launch_head_rows(const RowHeadParams& p, int bn, int sm_count, cudaStream_t s) {
    return p.f16 ? pick_rows<__half>(p, bn, sm_count, s) : pick_rows<__nv_bfloat16>(p, bn, sm_count, s);
}

namespace {
template <typename T, int R>
cudaError_t run_tokens_of(const TokenHeadParams& p, cudaStream_t s) {
    const size_t smem = sizeof(float) * R * ((p.k + 7) / 8 * 8);
    return launch_pdl(head_token_kernel<T, R>, dim3(head_token_blocks(p.cols)), dim3(32 * HEAD_TOKEN_WARPS), smem, s, p);
}
template <typename T>
cudaError_t pick_tokens_of(const TokenHeadParams& p, cudaStream_t s) {
    return p.rows == 1 ? run_tokens_of<T, 1>(p, s) : run_tokens_of<T, 2>(p, s);
}
}  // namespace

cudaError_t launch_head_tokens(const TokenHeadParams& p, cudaStream_t s) {
    return p.f16 ? pick_tokens_of<__half>(p, s) : pick_tokens_of<__nv_bfloat16>(p, s);
}

cudaError_t launch_head_join(const HeadJoinParams& p, cudaStream_t s) {
    return launch_pdl(head_join_kernel, dim3(static_cast<unsigned>((p.rows + HJ_ROWS - 1) / HJ_ROWS)), dim3(HJ_THREADS), 0, s, p);
}

cudaError_t launch_head_scale(const HeadScaleParams& p, cudaStream_t s) {
    return launch_pdl(head_scale_kernel, dim3(1), dim3(1024), 0, s, p);
}

cudaError_t launch_head_round(const HeadRoundParams& p, cudaStream_t s) {
    const long long items = (p.cols + 7) / 8 * p.rows, blocks = (items + 255) / 256;
    const dim3 grid(static_cast<unsigned>(blocks < 152 * 16 ? blocks : 152 * 16));
    return p.f16 ? launch_pdl(head_round_kernel<__half>, grid, dim3(256), 0, s, p)
                 : launch_pdl(head_round_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, p);
}

}  // namespace anvil
