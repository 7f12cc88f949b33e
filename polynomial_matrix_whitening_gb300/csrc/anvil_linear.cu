// anvil_linear.cu -- the linear layer's products for sm_103a: C = A B^T with 16-bit
// operands and fp32 accumulation on the 5th-generation tensor cores, and what follows the
// accumulator fused into the epilogue.
//
//   forward        z = x W^T + b,  y = act(z) + r
//   input's grad   dx = dz W
//   weight's grad  dW = dz^T x  (16 bit, or fp32, optionally added to what is there)
//
// Three kernels share the work.
//
// pair_gemm_kernel: clusters of two CTAs compute 256 x 256 output tiles with
// tcgen05.mma.cta_group::2; CTA rank r loads rows 128r.. of the tile's A operand and
// columns 128r.. of its B operand by TMA into a ring of five or six stages, and holds output rows
// 128r.. in its TMEM.  Two accumulators alternate, so a tile's epilogue overlaps the next
// tile's products.  Operands are taken in the order they are stored: K-major, or MN-major
// as 64 x 64 boxes, so no operand is ever transposed in memory.  The grid is persistent
// (one pair per two SMs), its tiles in groups of eight rows of tiles for the L2.  Tiles
// that would leave the last turn of the grid partly idle (or all of them, where they are
// few) are split along the contraction: the parts go to scratch in fp32 and
// finish_kernel adds them up, in order, and finishes the elements.  A backward pass's second
// product starts on the SMs that the first leaves idle in its last turn, its parts cut so
// that early and late pairs end together (8192 x 2816 x 768, squared-ReLU gradient and bias
// gradient included: 91 us one after the other, 77 so).
// What bounds it: at 16384 x 4096 x 4096 the products, within a few percent of the
// library's own rate; a tile narrower than 256 columns gains nothing (128 columns measured
// 660 SM cycles per 64-deep k-block against 560: a k-block's time is the L2 round trip of
// the stages in flight, not its bytes).  For short contractions the epilogue: the tensor
// pipe already takes about 96 of the 128 bytes per clock that shared memory gives, so every
// staged byte and every load instruction of the epilogue delays the products.
// fp32 results: the tensor cores add with truncation, a bias that grows with the length
// of the chain (about 1e-9 of the result per 16-deep step), so the product is taken in
// chains of 512 and the epilogue adds the chains up in registers, rounding to nearest.
//
// row_gemm_kernel: few rows (tokens).  The weight's 128-row blocks are the MMA's M side and
// the tokens its N side (16 to 128), so a weight is read once, and a cluster of up to eight
// CTAs splits the contraction, so that enough SMs read it; the partial accumulators are
// joined through distributed shared memory in rank order.  HBM bounds it where the weight
// is large (1 x 16384 x 4096: 23.3 us, 5.8 TB/s; 64 tokens 27), latency where it is small (16
// x 2816 x 768: 4.7 us), and from 128 tokens on the MMA's reads of its 128-row operand.
//
// token_kernel: one or two tokens and a small weight, without tensor cores.
//
// Every wait is bounded (anvil_device.cuh): one that gives up sets the device error word
// and an abort flag; loads in flight are waited for (bounded), the TMEM is freed and the
// CTA returns.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "anvil_device.cuh"
#include "anvil_linear.h"
#include "anvil_types.cuh"

namespace anvil {

namespace {

constexpr int CTA_ROWS = 128;
constexpr int A_STAGE = CTA_ROWS * 128; // 16 KB: this CTA's A rows of a k-block
constexpr int EPI_GROUPS = 4;           // epilogue warp groups, one per quarter of the columns
constexpr int EPI_WARP0 = 4;            // warps 4-19; warp 1: MMA issuer and TMEM owner; warps 0 and 2: TMA producers
constexpr int PRODUCERS = 2;
constexpr int PAIR_THREADS = 32 * (EPI_WARP0 + 4 * EPI_GROUPS);
constexpr int CHAIN_KB = 8;             // k-blocks of one chain of an fp32 result (512 deep)
constexpr int RASTER_ROWS = 8;          // rows of tiles per raster group

// 32 lanes x 16 or 8 consecutive fp32 columns of TMEM (as tmem_ld_32x32b_x32).
__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// kind::f16 instruction descriptor with fp32 accumulation; the operands' type is both
// bf16 (1) or both fp16 (0).
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool a_mn, bool b_mn, bool f16) {
    const uint32_t fmt = f16 ? 0u : 1u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// 1 / v to 1 ulp for v from 1 on (0 from 2^126 on).
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 2^v (a relative error of 2^-22; the subnormal results too).
__device__ __forceinline__ float power2(float v) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Phi(z), the normal distribution, and e = exp(-z^2/2).  Phi(-|z|) = e m(|z|) with m(a) =
// exp(a^2/2) erfc(a / sqrt 2) / 2, which falls slowly: m = t P(t), t = 1 / (1 + 0.305 a), P the
// polynomial of degree 7 of the least largest relative error over 0 <= a <= 16 (1.4e-7; fitted
// by iterated weighted least squares).  So the tail has a relative error of (48 + 2 z^2) 2^-24 at
// most, the exponential's own growth with its argument included, as far down as e reaches.
__device__ __forceinline__ float normal_cdf(float z, float* e) {
    const float t = reciprocal(fmaf(0.305f, fabsf(z), 1.f));
    float q = fmaf(t, 0.036033929f, -0.150315657f);
    q = fmaf(t, q, 0.181285652f);
    q = fmaf(t, q, -0.0340613788f);
    q = fmaf(t, q, 0.119038255f);
    q = fmaf(t, q, 0.103994657f);
    q = fmaf(t, q, 0.122379342f);
    q = fmaf(t, q, 0.121645144f);
    *e = power2(z * (z * -0.72134752044448170f));  // log2(e) / 2
    const float tail = t * q * *e;
    return z < 0.f ? tail : 1.f - tail;
}

// s = 1 / (1 + e^-u) and c = 1 - s for a u of z's sign, both to their relative accuracy: from
// e = e^-|u|, so that the divisor stays between 1 and 2 (1 + e^-u passes 2^126, where the
// reciprocal is 0).
__device__ __forceinline__ void sigmoid(float z, float e, float* s, float* c) {
    const float r = reciprocal(1.f + e);
    *s = z < 0.f ? e * r : r;
    *c = z < 0.f ? r : e * r;
}
// SiLU: u = z.  tanh-GELU is z sigmoid(u) with u = 2 sqrt(2/pi) (z + 0.044715 z^3).  Both e^-|u|
// with log2(e) in the factors.
__device__ __forceinline__ float silu_exp(float z) { return power2(fabsf(z) * -1.4426950408889634f); }
__device__ __forceinline__ float gelu_tanh_exp(float z, float zz) {
    return power2(fabsf(z) * fmaf(-0.10294324f, zz, -2.3022082f));
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.f ? 0.f : z;
    if constexpr (ACT == ACT_RELU2) return z < 0.f ? 0.f : z * z;
    if constexpr (ACT == ACT_GELU) {
        float e;
        return z * normal_cdf(z, &e);
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        float s, c;
        sigmoid(z, gelu_tanh_exp(z, z * z), &s, &c);
        return z * s;  // z (1 + tanh(u / 2)) / 2
    }
    if constexpr (ACT == ACT_SILU) {
        float s, c;
        sigmoid(z, silu_exp(z), &s, &c);
        return z * s;
    }
    return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;  // (NaN: NaN, as forward)
    if constexpr (ACT == ACT_RELU2) return z < 0.f ? 0.f : 2.f * z;
    if constexpr (ACT == ACT_GELU) {
        float e;
        const float c = normal_cdf(z, &e);
        return fmaf(z * 0.3989422804014327f, e, c);
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float zz = z * z, du = fmaf(0.21406451f, zz, 1.5957691f);  // du/dz
        float s, c;
        sigmoid(z, gelu_tanh_exp(z, zz), &s, &c);
        const float sc = s * c;
        return sc == 0.f ? s : s + z * sc * du;  // far out du overflows, and its factor is 0 long before
    }
    if constexpr (ACT == ACT_SILU) {
        float s, c;
        sigmoid(z, silu_exp(z), &s, &c);
        return s * (1.f + z * c);
    }
    return 1.f;
}
// The activation of N values, the choice made once.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
#define ANVIL_ACT_CASE(A)                                         \
    case A:                                                       \
        _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = act_value<A>(v[i]); \
        break
    switch (act) {
        ANVIL_ACT_CASE(ACT_RELU);
        ANVIL_ACT_CASE(ACT_RELU2);
        ANVIL_ACT_CASE(ACT_GELU);
        ANVIL_ACT_CASE(ACT_GELU_TANH);
        ANVIL_ACT_CASE(ACT_SILU);
        default: break;
    }
#undef ANVIL_ACT_CASE
}

// N bias values from column col0 (those at `cols` and beyond read as 0) added to v.
template <typename T, int N>
__device__ __forceinline__ void add_bias(const GemmEpilogue& e, int col0, int cols, float (&v)[N]) {
    const bool vec = col0 + N <= cols && !(reinterpret_cast<uintptr_t>(e.bias) & 15);
    if (e.bias_f32) {
        const float* b = static_cast<const float*>(e.bias) + col0;
        if (vec) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(b + i);
                v[i] += f.x;
                v[i + 1] += f.y;
                v[i + 2] += f.z;
                v[i + 3] += f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += col0 + i < cols ? b[i] : 0.f;
        }
    } else {
        const T* b = static_cast<const T*>(e.bias) + col0;
        if (vec) {
#pragma unroll
            for (int i = 0; i < N; i += 8) {
                float f[8];
                Elem<T>::unpack(*reinterpret_cast<const uint4*>(b + i), f);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[i + k] += f[k];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += col0 + i < cols ? Elem<T>::load(b[i]) : 0.f;
        }
    }
}

// ---------------------------------------------------------------- the pair kernel
constexpr int BN = PAIR_COLS;
constexpr int B_STAGE = BN / 2 * 128;  // 16 KB: this CTA's half of the B columns of a k-block
constexpr int STAGE = A_STAGE + B_STAGE;
constexpr int EPI_COLS = BN / EPI_GROUPS;  // 64
// The epilogue's staging boxes, one per group: 128 rows of W bytes, 16-byte chunk j of row r at
// the chunk the tensor maps' swizzle gives it.  W = 128 takes a group's 64 columns of 16-bit
// results at once; W = 64 takes them by halves and leaves the room of one more stage.
template <int W>
struct Staging {
    static constexpr int BOX = CTA_ROWS * W;
    static constexpr int STAGES = W == 128 ? 5 : 6;
    static constexpr int SMEM = STAGES * STAGE + EPI_GROUPS * BOX + 1024;  // + alignment slack
    static __device__ __forceinline__ uint32_t addr(uint32_t box, int r, int j) {
        return box + static_cast<uint32_t>(W == 128 ? r * 128 + ((j ^ (r & 7)) << 4) : r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
    }
};
constexpr uint32_t PAIR_TMEM = 2 * BN;

// Tile t: groups of RASTER_ROWS rows of tiles, column by column inside a group, so that the
// pairs running at one time share operand panels.
__device__ __forceinline__ void tile_at(int t, int tiles_r, int tiles_c, int* tr, int* tc) {
    const int per = RASTER_ROWS * tiles_c;
    const int g = t / per;
    const int rows = min(RASTER_ROWS, tiles_r - g * RASTER_ROWS);
    const int q = t - g * per;
    *tc = q / rows;
    *tr = g * RASTER_ROWS + (q - *tc * rows);
}

// Work unit u: a whole tile, or one part of a tail tile (part: its place in the scratch); no
// work (nkb = 0) where a turn of the tail has none left for its pair.
struct Unit {
    int tr, tc, part, kb0, nkb;
};
__device__ __forceinline__ Unit unit_of(const PairGemmParams& p, int u) {
    Unit r;
    const TileSplit& s = p.split;
    const int all = (p.k + GEMM_BK - 1) / GEMM_BK;
    int t = u;
    r.part = -1;
    r.kb0 = 0;
    r.nkb = all;
    if (u >= s.whole) {
        const int turn = (u - s.whole) / s.pairs, pair = (u - s.whole) - turn * s.pairs;
        const bool first = pair < s.early;
        const int parts = first ? s.sa : s.sb, kb = first ? s.kba : s.kbb;
        const int tiles = first ? s.tiles_a : p.tiles_r * p.tiles_c - s.whole - s.tiles_a;
        const int i = first ? turn * s.early + pair : turn * (s.pairs - s.early) + pair - s.early;
        const int q = i / parts;
        r.part = first ? i : s.tiles_a * s.sa + i;
        t = s.whole + (first ? q : s.tiles_a + q);
        r.kb0 = (i - q * parts) * kb;
        r.nkb = q < tiles ? max(0, min(kb, all - r.kb0)) : 0;
        if (q >= tiles) t = 0;
    }
    tile_at(t, p.tiles_r, p.tiles_c, &r.tr, &r.tc);
    return r;
}

// Results that TMA cannot store: the 32 box rows of this warp to global memory, neighbouring lanes
// on neighbouring elements, eight rows in flight.
template <typename E, int W>
__device__ __forceinline__ void box_to_rows(uint32_t box, E* dst, long long ld, int row0, int col0, int rows, int cols,
                                            int quad, int lane) {
    constexpr int C = W / sizeof(E);           // columns of a box
    constexpr int H = C > 32 ? C / 32 : 1;     // elements per lane of a box row
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += 8) {
        E v[8][H];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int c = C < 32 ? lane % C : h * 32 + lane;
                const int b = c * static_cast<int>(sizeof(E));
                const uint32_t a = Staging<W>::addr(box, quad * 32 + i0 + i, b / 16) + b % 16;
                if constexpr (sizeof(E) == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v[i][h]) : "r"(a) : "memory");
                else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[i][h]) : "r"(a) : "memory");
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int r = row0 + quad * 32 + i0 + i, c = h * 32 + lane;
                if (r < rows && (C >= 32 || lane < C) && col0 + c < cols) dst[static_cast<size_t>(r) * ld + col0 + c] = v[i][h];
            }
    }
}
// A residual or gradient whose rows are not 16-byte aligned (W = 128 then), the same way back.
template <typename E>
__device__ __forceinline__ void rows_to_box(uint32_t box, const E* src, long long ld, int row0, int col0, int rows,
                                            int cols, int quad, int lane) {
    constexpr int H = 128 / sizeof(E) / 32;
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += 8) {
        E v[8][H];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int r = row0 + quad * 32 + i0 + i, c = col0 + h * 32 + lane;
                v[i][h] = r < rows && c < cols ? src[static_cast<size_t>(r) * ld + c] : E(0);
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int c = h * 32 + lane;
                const int b = c * static_cast<int>(sizeof(E));
                const uint32_t a = Staging<128>::addr(box, quad * 32 + i0 + i, b / 16) + b % 16;
                if constexpr (sizeof(E) == 2) sts16(a, v[i][h]);
                else asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v[i][h]) : "memory");
            }
    }
}

// Per-thread epilogue state of one group (128 threads, one staging box).
struct EpiState {
    uint32_t box;        // shared address of the group's box
    uint64_t* in_bar;    // the barrier of its input loads
    int r, quad, lane, grp;
    bool leader;
    bool fail;
    int loads;           // input loads armed (parity of the barrier)
};

// The box may be written: its last store has been read.
__device__ __forceinline__ void box_free(const EpiState& x) {
    if (x.leader) bulk_wait_read_all();
    named_barrier_sync(1 + x.grp, 128);
}

__device__ __forceinline__ void tma_store_box(const CUtensorMap* tm, uint32_t box, int col, int row) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tm), "r"(box),
                 "r"(col), "r"(row), "r"(0)
                 : "memory");
}

// Sends the box out: by TMA (the group's leader, after every thread's writes), or by the
// warps themselves, each its own rows.  A tensor-map store is clipped to the map's width by 16-byte
// pieces (measured: a row of 97 16-bit elements has 104 written), so a box with a row end inside a
// piece is the warps' too: the bytes after it are not the result's.
template <typename E, int W>
__device__ __forceinline__ void send_box(const EpiState& x, const CUtensorMap* tm, int by_tma, void* dst, long long ld,
                                         int row0, int col0, int rows, int cols) {
    constexpr int C = W / sizeof(E), PIECE = 16 / sizeof(E);
    const bool cut = cols % PIECE != 0 && col0 < cols && col0 + C > cols;
    if ((W == 64 || by_tma) && !cut) {
        fence_proxy_async_smem();
        named_barrier_sync(1 + x.grp, 128);
        if (x.leader) {
            if (row0 < rows && col0 < cols) tma_store_box(tm, x.box, col0, row0);
            bulk_commit_group();
        }
    } else {
        __syncwarp();
        box_to_rows<E, W>(x.box, static_cast<E*>(dst), ld, row0, col0, rows, cols, x.quad, x.lane);
        fence_proxy_async_smem();  // before an input load into the box
        __syncwarp();
    }
}

template <int W>
__device__ __forceinline__ void arm_input(EpiState& x, const CUtensorMap* tm, int col0, int row0) {
    if (x.leader) {
        mbar_arrive_expect_tx(x.in_bar, Staging<W>::BOX);
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(x.box),
            "l"(tm), "r"(smem_u32(x.in_bar)), "r"(col0), "r"(row0), "r"(0)
            : "memory");
    }
    ++x.loads;
}
__device__ __forceinline__ void wait_input(EpiState& x, unsigned* err) {
    if (!mbar_wait(x.in_bar, static_cast<uint32_t>(x.loads - 1) & 1u, err)) x.fail = true;
}

// The accumulator is read: its next products may overwrite it.  That order rests on the loads'
// completion, not on the arrival: every lane has passed tcgen05.wait::ld (tmem_ld_* end with it),
// after which the values are in registers and no write can reach them, and __syncwarp joins the
// lanes before one of them arrives.  So the arrival may be relaxed, and orders nothing else: with
// release semantics it waited about 2000 cycles for the warp's shared-memory writes to be visible
// to the whole cluster, which nothing needs.
__device__ __forceinline__ void release_acc(const EpiState& x, uint32_t tempty) {
    tc_fence_before();
    __syncwarp();
    if (x.lane == 0) asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(tempty) : "memory");
}

// Whether a whole 16-bit tile's residual comes by TMA ahead of the accumulator: not where z
// takes the box first.
__device__ __forceinline__ bool early_input(const PairGemmParams& p) { return p.epi.in && p.in_tma && !p.epi.z; }

// The 16-bit epilogue of this group's quarter of a tile: z first where it is stored, then y
// (the accumulator is read again: TMEM is not what bounds it).
template <typename T, int W>
__device__ __forceinline__ void epilogue_16(const PairGemmParams& p, EpiState& x, uint32_t tacc, uint32_t tempty, int row0,
                                            int col0) {
    const GemmEpilogue& e = p.epi;
    const bool early = early_input(p);
    constexpr int COLS = W / 2, N = EPI_COLS / COLS;  // columns of a box, boxes
#pragma unroll 1
    for (int step = e.z ? 0 : N; step < 2 * N; ++step) {  // z's boxes, y's boxes
        const bool final = step >= N;
        const int from = step % N * COLS, col = col0 + from;
        const bool armed = early && step == N;
        if (armed) wait_input(x, p.err);
        else box_free(x);
        if (final && e.in && !armed) {
            if (W == 64 || p.in_tma) {
                arm_input<W>(x, &p.tm_in, col, row0);
                wait_input(x, p.err);
            } else {
                rows_to_box<uint16_t>(x.box, static_cast<const uint16_t*>(e.in), e.ldin, row0, col, p.rows, p.cols, x.quad,
                                      x.lane);
                __syncwarp();
            }
        }
#pragma unroll 1
        for (int c = 0; c < COLS / 16; ++c) {
            float v[16];
            tmem_ld_16(tacc + from + c * 16, v);
            if (e.bias) add_bias<T, 16>(e, col + c * 16, p.cols, v);
            if (final) act_values<16>(e.act, v);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t a = Staging<W>::addr(x.box, x.r, c * 2 + j);
                if (final && e.in) {
                    float f[8];
                    Elem<T>::unpack(lds128(a), f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[8 * j + i] += f[i];
                }
                sts128(a, Elem<T>::pack(v + 8 * j));
            }
        }
        if (step == 2 * N - 1) release_acc(x, tempty);
        if (final) send_box<uint16_t, W>(x, &p.tm_out, p.out_tma, e.out, e.ldout, row0, col, p.rows, p.cols);
        else send_box<uint16_t, W>(x, &p.tm_z, p.z_tma, e.z, e.ldz, row0, col, p.rows, p.cols);
    }
}

// A box of fp32 columns of this thread's row: to the scratch of split `part`, or
// to the fp32 result (with what it held).
template <int W>
__device__ __forceinline__ void store_f32(const PairGemmParams& p, EpiState& x, const float* v, int part, int lrow, int lcol,
                                          int row0, int col0) {
    const GemmEpilogue& e = p.epi;
    const bool in = e.in && part < 0;
    box_free(x);
    if (in) {
        if (W == 64 || p.in_tma) {
            arm_input<W>(x, &p.tm_in, col0, row0);
            wait_input(x, p.err);
        } else {
            rows_to_box<uint32_t>(x.box, static_cast<const uint32_t*>(e.in), e.ldin, row0, col0, p.rows, p.cols, x.quad, x.lane);
            __syncwarp();
        }
    }
#pragma unroll
    for (int j = 0; j < W / 16; ++j) {
        const uint32_t a = Staging<W>::addr(x.box, x.r, j);
        float f[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
        if (in) {
            float o[4];
            Elem<float>::unpack(lds128(a), o);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] += o[i];
        }
        sts128(a, Elem<float>::pack(f));
    }
    if (part >= 0) {
        fence_proxy_async_smem();
        named_barrier_sync(1 + x.grp, 128);
        if (x.leader) {
            tma_store_box(&p.tm_part, x.box, lcol, part * PAIR_ROWS + lrow);
            bulk_commit_group();
        }
    } else {
        send_box<uint32_t, W>(x, &p.tm_out, p.out_tma, e.out, e.ldout, row0, col0, p.rows, p.cols);
    }
}

// T: type of 16-bit results (float: fp32 results, taken in chains of CHAIN_KB k-blocks)
template <typename T, int W>
__global__ void __launch_bounds__(PAIR_THREADS, 1) pair_gemm_kernel(const __grid_constant__ PairGemmParams p) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int STAGES = Staging<W>::STAGES, COLS4 = W / 4;  // fp32 columns of a box
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[STAGES];
    __shared__ __align__(8) uint64_t empty_bar[STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[2];
    __shared__ __align__(8) uint64_t tempty_bar[2];
    __shared__ __align__(8) uint64_t in_bar[EPI_GROUPS];
    __shared__ __align__(8) uint64_t mma_done_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int aborted;
    __shared__ volatile int armed[STAGES];  // 1 + the k-block last loaded into each stage (0: none)

    if (!p.overlap_next) pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0 = leader (issues the MMAs)
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int units = p.units;
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
            armed[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], 2 * 4 * EPI_GROUPS);  // each epilogue warp of both CTAs
        }
        for (int g = 0; g < EPI_GROUPS; ++g) mbar_init(&in_bar[g], 1);
        mbar_init(&mma_done_bar, 1);
        fence_mbar_init();
        aborted = 0;
        tma_prefetch_desc(&p.tm_a);
        tma_prefetch_desc(&p.tm_b);
    }
    if (warp == 1) tmem_alloc_pair(&tmem_slot, PAIR_TMEM);
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    // The two products of a backward pass read nothing of each other's: the first lets the
    // second start once the kernels before both have ended, and the second's pairs run on the
    // SMs that the first leaves idle in its last turn.  The second ends after the first, so
    // that what waits for it has both.
    if (!p.overlap_previous) pdl_wait_previous();
    if (p.overlap_next) pdl_allow_next();
    const uint32_t tmem = tmem_slot;

    if (warp == 0 || warp == 2) {
        if (lane == 0) {
            // ---------------- TMA producers: arming a stage and issuing its two loads takes one
            // thread about 500 cycles, as long as its products, so two take turns
            int it = 0;
            const int mine = warp / 2;
            Unit next = unit_of(p, pair < units ? pair : 0);
            for (int u = pair; u < units; u += npairs) {
                const Unit t = next;
                bool looked = u + npairs >= units;  // the next unit's place: its divisions run while this one's loads do
                const int arow = t.tr * PAIR_ROWS + CTA_ROWS * static_cast<int>(rank);
                const int brow = t.tc * BN + BN / 2 * static_cast<int>(rank);
                bool ok = true;
                for (int kb = t.kb0; kb < t.kb0 + t.nkb; ++kb, ++it) {
                    if (it % PRODUCERS != mine) continue;
                    const int s = it % STAGES;
                    if (!mbar_wait(&empty_bar[s], ((it / STAGES) & 1) ^ 1, p.err)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full_bar[s], 2 * STAGE);
                    armed[s] = it + 1;
                    const uint32_t fb = map_to_rank(&full_bar[s], 0);
                    uint8_t* sa = smem + s * STAGE;
                    uint8_t* sb = sa + A_STAGE;
                    const int kc = kb * GEMM_BK;
                    if (p.a_mn) {
                        tma_load_3d_pair(sa, &p.tm_a, fb, arow, kc, 0);
                        tma_load_3d_pair(sa + 8192, &p.tm_a, fb, arow + 64, kc, 0);
                    } else {
                        tma_load_3d_pair(sa, &p.tm_a, fb, kc, arow, 0);
                    }
                    if (p.b_mn) {
                        tma_load_3d_pair(sb, &p.tm_b, fb, brow, kc, 0);
                        tma_load_3d_pair(sb + 8192, &p.tm_b, fb, brow + 64, kc, 0);
                    } else {
                        tma_load_3d_pair(sb, &p.tm_b, fb, kc, brow, 0);
                    }
                    if (!looked) {
                        looked = true;
                        next = unit_of(p, u + npairs);
                    }
                }
                if (!looked) next = unit_of(p, u + npairs);
                if (!ok) {
                    aborted = 1;
                    break;
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMA issuer (leader CTA): the next stage's barrier is tested while
            // this k-block's MMAs run, and waited for only when that test found it not loaded
            const uint32_t stage0 = smem_u32(smem);
            const uint32_t idesc = idesc_16(PAIR_ROWS, BN, p.a_mn, p.b_mn, p.f16);
            const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;
            const uint32_t a_lbo = p.a_mn ? 8192 : 16, b_lbo = p.b_mn ? 8192 : 16;
            const int whole_kb = (p.k + GEMM_BK - 1) / GEMM_BK;
            int s = 0, acc = 0;
            uint32_t ph = 0;
            bool ready = false, ok = true;
            for (int u = pair; u < units && ok; u += npairs) {
                const int nkb = u < p.split.whole ? whole_kb : unit_of(p, u).nkb;
                for (int c0 = 0; c0 < nkb && ok; c0 += F32 ? CHAIN_KB : nkb, ++acc) {
                    const int cn = F32 ? min(CHAIN_KB, nkb - c0) : nkb;
                    const int ab = acc & 1;
                    if (!mbar_wait(&tempty_bar[ab], ((acc >> 1) & 1) ^ 1, p.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t dacc = tmem + static_cast<uint32_t>(ab * BN);
                    for (int kb = 0; kb < cn; ++kb) {
                        if (!ready && !mbar_wait(&full_bar[s], ph, p.err)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a0 = stage0 + static_cast<uint32_t>(s * STAGE);
                        const uint32_t a_lo = sw128_desc_lo(a0, a_lbo), b_lo = sw128_desc_lo(a0 + A_STAGE, b_lbo);
#pragma unroll
                        for (int kk = 0; kk < GEMM_BK / 16; ++kk)
                            umma_bf16_pair(dacc, sw128_desc(a_lo + kk * a_step), sw128_desc(b_lo + kk * b_step), idesc,
                                           (kb | kk) != 0 ? 1u : 0u);
                        const int s_next = s + 1 == STAGES ? 0 : s + 1;
                        const uint32_t ph_next = s_next == 0 ? ph ^ 1u : ph;
                        ready = mbar_test_wait(smem_u32(&full_bar[s_next]), ph_next);
                        umma_commit_pair(&empty_bar[s], 3);  // frees stage s in both CTAs
                        s = s_next;
                        ph = ph_next;
                    }
                    if (ok) umma_commit_pair(&tfull_bar[ab], 3);  // accumulator complete in both CTAs
                }
            }
            if (!ok) aborted = 1;
            umma_commit_pair(&mma_done_bar, 3);
            mbar_wait(&mma_done_bar, 0, p.err);
        } else if (lane == 0) {
            mbar_wait(&mma_done_bar, 0, p.err);  // peer: the leader's MMAs write this CTA's TMEM
        }
    } else if (warp >= EPI_WARP0) {
        // ---------------- epilogue: TMEM lane quadrant = warp % 4
        EpiState x;
        x.quad = warp & 3;
        x.grp = (warp - EPI_WARP0) >> 2;
        x.lane = lane;
        x.r = x.quad * 32 + lane;
        x.leader = x.quad == 0 && lane == 0;
        x.box = smem_u32(smem + STAGES * STAGE + x.grp * Staging<W>::BOX);
        x.in_bar = &in_bar[x.grp];
        x.fail = false;
        x.loads = 0;
        const uint32_t te[2] = {map_to_rank(&tempty_bar[0], 0), map_to_rank(&tempty_bar[1], 0)};
        const int lrow = CTA_ROWS * static_cast<int>(rank), lcol = EPI_COLS * x.grp;  // within the tile
        int acc = 0;
        for (int u = pair; u < units; u += npairs) {
            // the group stops together once any wait of any role gave up
            if (named_barrier_or(1 + x.grp, 128, x.fail || aborted)) {
                aborted = 1;
                break;
            }
            const Unit t = unit_of(p, u);
            if (t.nkb == 0) continue;
            const int row0 = t.tr * PAIR_ROWS + lrow;
            const int col0 = t.tc * BN + lcol;
            const uint32_t tlane = tmem + (static_cast<uint32_t>(x.quad * 32) << 16) + static_cast<uint32_t>(lcol);
            if constexpr (F32) {
                float sum[EPI_COLS];
#pragma unroll
                for (int i = 0; i < EPI_COLS; ++i) sum[i] = 0.f;
                for (int c0 = 0; c0 < t.nkb; c0 += CHAIN_KB, ++acc) {
                    const int ab = acc & 1;
                    if (!mbar_wait(&tfull_bar[ab], (acc >> 1) & 1, p.err)) x.fail = true;
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < EPI_COLS / 16; ++q) {
                        float v[16];
                        tmem_ld_16(tlane + ab * BN + q * 16, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[q * 16 + i] += v[i];
                    }
                    release_acc(x, te[ab]);
                }
#pragma unroll
                for (int q = 0; q < EPI_COLS / COLS4; ++q)
                    store_f32<W>(p, x, sum + COLS4 * q, t.part, lrow, lcol + COLS4 * q, row0, col0 + COLS4 * q);
            } else {
                const int ab = acc & 1;
                if (t.part < 0 && early_input(p)) {
                    // the residual, once the box's earlier store has been read
                    if (x.leader) bulk_wait_read_all();
                    arm_input<W>(x, &p.tm_in, col0, row0);
                }
                if (!mbar_wait(&tfull_bar[ab], (acc >> 1) & 1, p.err)) x.fail = true;
                tc_fence_after();
                if (t.part < 0) {
                    epilogue_16<T, W>(p, x, tlane + ab * BN, te[ab], row0, col0);
                } else {
#pragma unroll 1
                    for (int q = 0; q < EPI_COLS / COLS4; ++q) {
                        float v[COLS4];
                        if constexpr (COLS4 == 32) tmem_ld_32x32b_x32(tlane + ab * BN + q * COLS4, v);
                        else tmem_ld_16(tlane + ab * BN + q * COLS4, v);
                        if (q == EPI_COLS / COLS4 - 1) release_acc(x, te[ab]);
                        store_f32<W>(p, x, v, t.part, lrow, lcol + COLS4 * q, row0, col0 + COLS4 * q);
                    }
                }
                ++acc;
            }
        }
        if (x.leader) {
            bulk_wait_read_all();  // the group's last store has read its box
            if (x.loads) mbar_wait(x.in_bar, static_cast<uint32_t>(x.loads - 1) & 1u, p.err);
        }
    }

    __syncthreads();
    if (aborted && warp == 0 && lane == 0 && rank == 0) {
        // the pair's loads in flight land before its shared memory goes away
        for (int s = 0; s < STAGES; ++s)
            if (armed[s]) mbar_wait(&full_bar[s], ((armed[s] - 1) / STAGES) & 1, p.err);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, PAIR_TMEM);
    if (p.overlap_previous) pdl_wait_previous();
}

// The tail tiles of pair_gemm_kernel: the parts of each element, in order, then what follows
// the accumulator.  A block takes 16 rows of a tile, a thread one column of them, so that
// neighbouring lanes are neighbouring elements whatever the arrays' alignment.
constexpr int FINISH_THREADS = PAIR_COLS;
constexpr int TAIL_ROWS = 16, TAIL_BLOCKS = PAIR_ROWS / TAIL_ROWS;
template <typename T>
__device__ __forceinline__ void tail_sum(const TailSumParams& p, int block) {
    const GemmEpilogue& e = p.epi;
    const int tile = block / TAIL_BLOCKS, r0 = block % TAIL_BLOCKS * TAIL_ROWS;
    int tr, tc;
    tile_at(p.split.whole + tile, p.tiles_r, p.tiles_c, &tr, &tc);
    const int col = tc * PAIR_COLS + threadIdx.x;
    const int rows = min(TAIL_ROWS, p.rows - tr * PAIR_ROWS - r0);  // of this block that exist
    const long long row = static_cast<long long>(tr) * PAIR_ROWS + r0;
    if (rows <= 0 || col >= p.cols) return;  // (the block's other threads wait for the parts)
    pdl_wait_previous();  // (the product may have let this kernel start before what came before it had ended)
    float bias = 0.f;
    if constexpr (sizeof(T) == 2) {
        if (e.bias)
            bias = e.bias_f32 ? static_cast<const float*>(e.bias)[col] : Elem<T>::load(static_cast<const T*>(e.bias)[col]);
    }
    const bool first = tile < p.split.tiles_a;
    const int splits = first ? p.split.sa : p.split.sb;
    const int part0 = first ? tile * splits : p.split.tiles_a * p.split.sa + (tile - p.split.tiles_a) * splits;
    const float* part = p.part + (static_cast<size_t>(part0) * PAIR_ROWS + r0) * PAIR_COLS + threadIdx.x;
    float v[TAIL_ROWS], in[TAIL_ROWS];
#pragma unroll
    for (int i = 0; i < TAIL_ROWS; ++i) {
        v[i] = __ldcs(part + i * PAIR_COLS);
        in[i] = e.in && i < rows ? Elem<T>::load(static_cast<const T*>(e.in)[(row + i) * e.ldin + col]) : 0.f;
    }
    for (int s = 1; s < splits; ++s) {
        part += static_cast<size_t>(PAIR_ROWS) * PAIR_COLS;
#pragma unroll
        for (int i = 0; i < TAIL_ROWS; ++i) v[i] += __ldcs(part + i * PAIR_COLS);
    }
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < TAIL_ROWS; ++i) v[i] += bias;
        if (e.z) {
#pragma unroll
            for (int i = 0; i < TAIL_ROWS; ++i)
                if (i < rows) static_cast<T*>(e.z)[(row + i) * e.ldz + col] = Elem<T>::store(v[i]);
        }
        act_values<TAIL_ROWS>(e.act, v);
    }
#pragma unroll
    for (int i = 0; i < TAIL_ROWS; ++i)
        if (i < rows) static_cast<T*>(e.out)[(row + i) * e.ldout + col] = Elem<T>::store(v[i] + in[i]);
}

// 32 columns of a bias gradient: the blocks' sums, every eighth of them per warp, in order.
constexpr int CS_COLS = 32, CS_LANES = FINISH_THREADS / CS_COLS;
__device__ __forceinline__ void column_sum(const ColumnSumParams& p, int block) {
    __shared__ float s[CS_LANES][CS_COLS];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = block * CS_COLS + x;
    pdl_wait_previous();
    float a = 0.f;
    if (c < p.cols) {
#pragma unroll 8
        for (int b = y; b < p.blocks; b += CS_LANES) a += p.part[static_cast<size_t>(b) * p.cols + c];
    }
    s[y][x] = a;
    __syncthreads();
    if (y == 0 && c < p.cols) {
        for (int k = 1; k < CS_LANES; ++k) a += s[k][x];
        p.out[c] = p.accumulate ? p.out[c] + a : a;
    }
}

// Everything that is added up after the products: one launch (T: type of 16-bit results).
template <typename T>
__global__ void __launch_bounds__(FINISH_THREADS) finish_kernel(const __grid_constant__ FinishParams p) {
    pdl_allow_next();
    int b = blockIdx.x;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const TailSumParams& t = p.tail[j];
        const int blocks = t.tiles * TAIL_BLOCKS;
        if (b < blocks) {
            if (t.epi.out_f32) tail_sum<float>(t, b);
            else tail_sum<T>(t, b);
            return;
        }
        b -= blocks;
    }
    column_sum(p.bias, b);
}

// ---------------------------------------------------------------- few rows
constexpr int ROW_THREADS = 256;  // warp 1: MMA issuer and TMEM owner, warps 2-5: epilogue, warps 0, 6 and 7: TMA producers
constexpr int ROW_PRODUCERS = 3;
template <int BN>
struct RowShape {
    static constexpr int STAGE = A_STAGE + BN * 128;
    static constexpr int STAGES = BN <= 64 ? 8 : 6;
    // Two blocks per SM where there are more blocks than SMs: one's first loads and last stores
    // run beside the other's products (1 x 50304 x 768: 17.3 us, 20.6 with one; from 64 tokens
    // on the fewer stages cost more than that gives, 24 against 21).
    static constexpr int STAGES_OF_TWO = 110 * 1024 / STAGE;
    static constexpr int smem(int stages) { return stages * STAGE + 1024; }
    static constexpr uint32_t TMEM_COLS = BN < 32 ? 32 : BN;
    static_assert(BN * ROW_TILE_A * 4 <= STAGES * STAGE && STAGES_OF_TWO < STAGES, "the partial accumulator reuses the stages");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

// bias, activation, residual and stores of up to N rows (B's) of one column (A's row);
// neighbouring lanes are neighbouring columns.  The loads go out together.
template <typename T, int N>
__device__ __forceinline__ void finish_rows(const GemmEpilogue& e, float (&v)[N], float bias, long long row, int rows, int col) {
    float in[N];
    if (e.in) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            in[i] = i < rows ? Elem<T>::load(static_cast<const T*>(e.in)[(row + i) * e.ldin + col]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += bias;
    if (e.z) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < rows) static_cast<T*>(e.z)[(row + i) * e.ldz + col] = Elem<T>::store(v[i]);
    }
    act_values<N>(e.act, v);
    if (e.in) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += in[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < rows) static_cast<T*>(e.out)[(row + i) * e.ldout + col] = Elem<T>::store(v[i]);
}

template <typename T, int BN>
__global__ void __launch_bounds__(ROW_THREADS, 2) row_gemm_kernel(const __grid_constant__ RowGemmParams p) {
    using S = RowShape<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[S::STAGES];
    __shared__ __align__(8) uint64_t empty_bar[S::STAGES];
    __shared__ __align__(8) uint64_t done_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int aborted;
    __shared__ volatile int armed[S::STAGES];  // 1 + the k-block last loaded into each stage (0: none)

    pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % p.splits;  // rank in the cluster
    const int a0 = blockIdx.x / p.splits * ROW_TILE_A;
    const int b0 = blockIdx.y * BN;
    const int all = (p.k + GEMM_BK - 1) / GEMM_BK;
    const int kb0 = split * p.kb_per_split;
    const int nkb = max(0, min(p.kb_per_split, all - kb0));
    const int stages = p.stages;
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
            armed[s] = 0;
        }
        mbar_init(&done_bar, 1);
        fence_mbar_init();
        aborted = 0;
        tma_prefetch_desc(&p.tm_a);
        tma_prefetch_desc(&p.tm_b);
    }
    if (warp == 1) tmem_alloc(&tmem_slot, S::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait_previous();
    const uint32_t tmem = tmem_slot;

    if (warp == 0 || warp >= 6) {
        if (lane == 0) {
            const int mine = warp == 0 ? 0 : warp - 5;
            for (int it = mine; it < nkb; it += ROW_PRODUCERS) {
                const int s = it % stages;
                if (!mbar_wait(&empty_bar[s], ((it / stages) & 1) ^ 1, p.err)) {
                    aborted = 1;
                    break;
                }
                mbar_arrive_expect_tx(&full_bar[s], S::STAGE);
                armed[s] = it + 1;
                uint8_t* sa = smem + s * S::STAGE;
                const int kc = (kb0 + it) * GEMM_BK;
                if (p.a_mn) {
                    tma_load_3d(sa, &p.tm_a, &full_bar[s], a0, kc, 0);
                    tma_load_3d(sa + 8192, &p.tm_a, &full_bar[s], a0 + 64, kc, 0);
                } else {
                    tma_load_3d(sa, &p.tm_a, &full_bar[s], kc, a0, 0);
                }
                tma_load_3d(sa + A_STAGE, &p.tm_b, &full_bar[s], kc, b0, 0);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t stage0 = smem_u32(smem);
            const uint32_t idesc = idesc_16(ROW_TILE_A, BN, p.a_mn, false, p.f16);
            const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, a_lbo = p.a_mn ? 8192 : 16;
            int s = 0;
            uint32_t ph = 0;
            bool ready = false;
            for (int it = 0; it < nkb; ++it) {
                if (!ready && !mbar_wait(&full_bar[s], ph, p.err)) {
                    aborted = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = stage0 + static_cast<uint32_t>(s * S::STAGE);
                const uint32_t a_lo = sw128_desc_lo(sa, a_lbo), b_lo = sw128_desc_lo(sa + A_STAGE, 16);
#pragma unroll
                for (int kk = 0; kk < GEMM_BK / 16; ++kk)
                    umma_bf16(tmem, sw128_desc(a_lo + kk * a_step), sw128_desc(b_lo + kk * (32 >> 4)), idesc,
                              (it | kk) != 0 ? 1u : 0u);
                const int s_next = s + 1 == stages ? 0 : s + 1;
                const uint32_t ph_next = s_next == 0 ? ph ^ 1u : ph;
                ready = mbar_test_wait(smem_u32(&full_bar[s_next]), ph_next);
                umma_commit(&empty_bar[s]);
                s = s_next;
                ph = ph_next;
            }
            umma_commit(&done_bar);
            mbar_wait(&done_bar, 0, p.err);
        }
    } else {
        // ---------------- epilogue: thread = one row of A (one output column)
        const int quad = warp & 3;
        const int r = quad * 32 + lane;
        const int col = a0 + r;
        const bool live = col < p.na;
        const int nb = min(BN, p.nb - b0);
        const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        float bias = 0.f;
        if (live && p.epi.bias)
            bias = p.epi.bias_f32 ? static_cast<const float*>(p.epi.bias)[col] : Elem<T>::load(static_cast<const T*>(p.epi.bias)[col]);
        mbar_wait(&done_bar, 0, p.err);
        tc_fence_after();
        if (p.splits == 1) {
#pragma unroll 1
            for (int q = 0; q < nb; q += 8) {
                float v[8];
                tmem_ld_8(tlane + q, v);
                if (live) finish_rows<T, 8>(p.epi, v, bias, b0 + q, nb - q, col);
            }
        } else {
            // the partial accumulator, in place of the stages (which are done): four B rows of one
            // A row side by side, [BN / 4][128] of them
            float4* own = reinterpret_cast<float4*>(smem);
            const int quads = (nb + 3) / 4;
#pragma unroll 1
            for (int q = 0; q < quads; q += 2) {
                float v[8];
                tmem_ld_8(tlane + q * 4, v);
                own[q * ROW_TILE_A + r] = make_float4(v[0], v[1], v[2], v[3]);
                own[(q + 1) * ROW_TILE_A + r] = make_float4(v[4], v[5], v[6], v[7]);
            }
            __syncwarp();
            cluster_sync();
            // every CTA finishes its share of the B rows, two fours at a time, the parts added in
            // rank order (rows past nb are computed and not stored)
#pragma unroll 1
            for (int j = 2 * split; j < quads; j += 2 * p.splits) {
                const uint32_t mine = smem_u32(&own[j * ROW_TILE_A + r]);
                float4 f[8][2];  // every part on its way before the first is used
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    if (s >= p.splits) break;
                    uint32_t a;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(mine), "r"(s));
                    f[s][0] = ld_cluster_f4(a);
                    f[s][1] = ld_cluster_f4(a + 16 * ROW_TILE_A);
                }
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    if (s >= p.splits) break;
                    v[0] += f[s][0].x;
                    v[1] += f[s][0].y;
                    v[2] += f[s][0].z;
                    v[3] += f[s][0].w;
                    v[4] += f[s][1].x;
                    v[5] += f[s][1].y;
                    v[6] += f[s][1].z;
                    v[7] += f[s][1].w;
                }
                if (live) finish_rows<T, 8>(p.epi, v, bias, b0 + 4 * j, nb - 4 * j, col);
            }
            __syncwarp();
        }
        tc_fence_before();
    }
    __syncwarp();
    if (p.splits > 1) {
        if (warp < 2 || warp >= 6) cluster_sync();  // the first barrier of the epilogue warps above
        cluster_sync();                // no CTA leaves while its partial accumulator is read
    }
    __syncthreads();
    if (aborted && threadIdx.x == 0) {
        // the loads in flight land before the shared memory goes away
        for (int s = 0; s < stages; ++s)
            if (armed[s]) mbar_wait(&full_bar[s], ((armed[s] - 1) / stages) & 1, p.err);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, S::TMEM_COLS);
}

// ---------------------------------------------------------------- one or two tokens
// For small weights, where the latency of one load after another is what a call costs (1 x 2816
// x 768: 2.7 us; the row kernel, with its barriers, tensor memory and join: 4.4).  A warp takes
// WR weight rows (or a ks-th of the chunks of each) with eight loads of 16 bytes in flight per
// lane, the tokens wait in shared memory; fp32 FMAs on packed pairs, the lanes' sums joined by
// shuffles, the parts of a row through shared memory in order.
constexpr int TOKEN_THREADS = 256, TOKEN_WARPS = TOKEN_THREADS / 32;
template <typename T, int R, int WR>
__global__ void __launch_bounds__(TOKEN_THREADS) token_kernel(const TokenParams p, int ks) {
    constexpr int E = Elem<T>::VEC, U = 8 / WR;
    extern __shared__ __align__(16) uint8_t xs[];  // the tokens' whole chunks
    __shared__ float parts[TOKEN_WARPS][WR * R];
    pdl_allow_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % ks;
    const int col0 = (blockIdx.x * (TOKEN_WARPS / ks) + warp / ks) * WR;
    const T* w[WR];
#pragma unroll
    for (int i = 0; i < WR; ++i) w[i] = static_cast<const T*>(p.w) + static_cast<long long>(min(col0 + i, p.cols - 1)) * p.ldw;
    const int chunks = p.k / E;
    uint64_t acc[WR][R];
#pragma unroll
    for (int i = 0; i < WR; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[i][r] = 0;
    pdl_wait_previous();
    const uint32_t xa = smem_u32(xs);
    bool staged = false;
    for (int c0 = part * 32 + lane; c0 - lane < chunks; c0 += 32 * ks * U) {
        uint4 wr[U][WR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 * ks;
#pragma unroll
            for (int i = 0; i < WR; ++i) wr[u][i] = c < chunks ? ldg_stream(w[i] + c * E) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (!staged) {  // the tokens, while the first weights are on their way
            staged = true;
            for (int i = threadIdx.x; i < chunks * R; i += TOKEN_THREADS) {
                const int r = i / chunks, c = i - r * chunks;
                const T* x = static_cast<const T*>(p.x) + min(r, p.rows - 1) * p.ldx;
                sts128(xa + i * 16, reinterpret_cast<const uint4*>(x)[c]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 * ks;
            if (c >= chunks) break;
            uint64_t xv[R][E / 2];
#pragma unroll
            for (int r = 0; r < R; ++r) Elem<T>::unpack_pairs(lds128(xa + (r * chunks + c) * 16), xv[r]);
#pragma unroll
            for (int i = 0; i < WR; ++i) {
                uint64_t wv[E / 2];
                Elem<T>::unpack_pairs(wr[u][i], wv);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) acc[i][r] = f2_fma(wv[e], xv[r][e], acc[i][r]);
            }
        }
    }
    const bool tail = part == 0 && lane < p.k - chunks * E;  // the elements after the last whole chunk
    float v[WR][R];
#pragma unroll
    for (int i = 0; i < WR; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float lo, hi;
            f2_split(acc[i][r], &lo, &hi);
            v[i][r] = lo + hi;
            if (tail) v[i][r] = fmaf(Elem<T>::load(w[i][chunks * E + lane]), 
                                      Elem<T>::load(static_cast<const T*>(p.x)[min(r, p.rows - 1) * p.ldx + chunks * E + lane]), v[i][r]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[i][r] += __shfl_xor_sync(0xffffffffu, v[i][r], o);
        }
    if (ks > 1) {
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < WR; ++i)
#pragma unroll
                for (int r = 0; r < R; ++r) parts[warp][i * R + r] = v[i][r];
        }
        __syncthreads();
        if (part != 0) return;
#pragma unroll
        for (int i = 0; i < WR; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r)
                for (int q = 1; q < ks; ++q) v[i][r] += parts[warp + q][i * R + r];
    }
    // lane i * R + r finishes weight row i's value of token r
    float mine[1] = {0.f};
#pragma unroll
    for (int i = 0; i < WR; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane == i * R + r) mine[0] = v[i][r];
    const int col = col0 + lane / R, row = lane % R;
    if (lane >= WR * R || col >= p.cols || row >= p.rows) return;
    const GemmEpilogue& e = p.epi;
    if (e.bias) mine[0] += e.bias_f32 ? static_cast<const float*>(e.bias)[col] : Elem<T>::load(static_cast<const T*>(e.bias)[col]);
    if (e.z) static_cast<T*>(e.z)[row * e.ldz + col] = Elem<T>::store(mine[0]);
    act_values<1>(e.act, mine);
    if (e.in) mine[0] += Elem<T>::load(static_cast<const T*>(e.in)[row * e.ldin + col]);
    static_cast<T*>(e.out)[row * e.ldout + col] = Elem<T>::store(mine[0]);
}

// ---------------------------------------------------------------- around the products
// Eight columns per thread; the last chunk of a row may be partial.
__global__ void __launch_bounds__(256) repack_kernel(const __grid_constant__ RepackParams q) {
    const Repack& p = q.job[blockIdx.y];
    pdl_wait_previous();  // (the product starts after this kernel: its shared memory would take the L1 that the loads need)
    const long long chunks = (p.cols + 7) / 8;
    const long long total = chunks * p.rows;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long row = i / chunks;
        const int c = static_cast<int>(i - row * chunks) * 8;
        const uint16_t* s = p.src + row * p.lds + c;
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = c + e < p.cols && row < p.src_rows ? s[e] : 0u;
        *reinterpret_cast<uint4*>(p.dst + row * p.ldd + c) =
            make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}

// dz = dy act'(z), and the bias's gradient from the unrounded values.  dz itself is rounded once to
// the operands' type, because it is an operand: the tensor cores multiply 16-bit values.  Each
// element is off by 2^-8 of itself (fp16 2^-11) at most, which leaves a sum over many rows or
// columns off by less, relative to the root of its terms' squares: at 8192 x 2816 x 768 bf16 the
// gradients are 0.0023 off (norm) where fp32 dz and results rounded to bf16 give 0.0017.  A caller
// who needs more asks for two parts (what the rounding drops as a second operand, the products'
// contraction twice as long, W and x laid out twice: the call takes 140 us there instead of 80).
// In fp16 a dz beyond 65504 becomes infinite either way, and with it what it is added to.
constexpr int AG_LANES = 8;   // rows at a time per block: 32 threads x 8 columns each
constexpr int AG_UNROLL = 4;  // turns whose loads are in flight together
template <typename T, int ACT, bool VEC>
__global__ void __launch_bounds__(32 * AG_LANES, ACT_GRAD_BLOCKS) act_grad_kernel(const ActGradParams p) {
    __shared__ float sums[AG_LANES][ACT_GRAD_COLS];
    constexpr bool Z = ACT != ACT_NONE;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * ACT_GRAD_COLS + tx * 8;
    const T* dy = static_cast<const T*>(p.dy) + c;
    const T* z = static_cast<const T*>(p.z) + c;
    T* dz = static_cast<T*>(p.dz);
    pdl_allow_next();
    pdl_wait_previous();
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const long long r0 = static_cast<long long>(blockIdx.y) * p.rows_per_block;
    const long long r1 = min(r0 + p.rows_per_block, p.rows);
    if (c < p.cols) {
        auto fetch = [&](const T* q) {
            if constexpr (VEC) {
                return ldg_stream(q);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = c + e < p.cols ? __ldcs(reinterpret_cast<const uint16_t*>(q) + e) : 0u;
                return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
        };
        for (long long rb = r0 + ty; rb < r1; rb += AG_LANES * AG_UNROLL) {
            uint4 rg[AG_UNROLL], rz[AG_UNROLL];
#pragma unroll
            for (int k = 0; k < AG_UNROLL; ++k) {
                const long long r = rb + k * AG_LANES;
                rg[k] = r < r1 ? fetch(dy + r * p.lddy) : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (Z) rz[k] = r < r1 ? fetch(z + r * p.ldz) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < AG_UNROLL; ++k) {
                const long long r = rb + k * AG_LANES;
                float g[8];
                Elem<T>::unpack(rg[k], g);
                if constexpr (Z) {
                    float f[8];
                    Elem<T>::unpack(rz[k], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] *= act_slope<ACT>(f[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += g[e];
                if (dz && r < r1) {
                    const uint4 w = Elem<T>::pack(g);
                    *reinterpret_cast<uint4*>(dz + r * p.ldd + c) = w;
                    if (Z && p.two_parts) {
                        float h[8];
                        Elem<T>::unpack(w, h);
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = isfinite(h[e]) ? g[e] - h[e] : 0.f;
                        *reinterpret_cast<uint4*>(dz + r * p.ldd + p.ldd / 2 + c) = Elem<T>::pack(h);
                    }
                }
            }
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[ty][tx * 8 + e] = acc[e];
    __syncthreads();
    const int cc = blockIdx.x * ACT_GRAD_COLS + threadIdx.x;
    if (cc < p.cols) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < AG_LANES; ++k) s += sums[k][threadIdx.x];
        p.part[static_cast<size_t>(blockIdx.y) * p.cols + cc] = s;
    }
}

template <typename T, int W>
cudaError_t run_pair(const PairGemmParams& p, int sm_count, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(PAIR_THREADS);
    cfg.dynamicSmemBytes = Staging<W>::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const int most = sm_count / 2;
    cfg.gridDim = dim3(2 * (p.units < most ? p.units : most));
    return cudaLaunchKernelEx(&cfg, pair_gemm_kernel<T, W>, p);
}

template <typename T, int BN>
cudaError_t run_row(RowGemmParams p, int sm_count, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((p.na + ROW_TILE_A - 1) / ROW_TILE_A * p.splits, (p.nb + BN - 1) / BN);
    cfg.blockDim = dim3(ROW_THREADS);
    const bool more = BN <= ROW_TWO_TOKENS && static_cast<long long>(cfg.gridDim.x) * cfg.gridDim.y > sm_count;
    p.stages = more ? RowShape<BN>::STAGES_OF_TWO : RowShape<BN>::STAGES;
    cfg.dynamicSmemBytes = RowShape<BN>::smem(p.stages);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, row_gemm_kernel<T, BN>, p);
}

// Weight rows per warp: four where that still gives every SM sixteen warps, else fewer, then
// several warps per row, as long as every lane has a chunk.
template <typename T, int R>
cudaError_t run_tokens(const TokenParams& p, cudaStream_t s) {
    const int full = 152 * 2 * TOKEN_WARPS, chunks = p.k / Elem<T>::VEC;
    const int wr = p.cols >= 4 * full ? 4 : p.cols >= 2 * full ? 2 : 1;
    int ks = 1;
    while (ks < TOKEN_WARPS && static_cast<long long>(p.cols) * ks < full && chunks >= 64 * ks) ks *= 2;
    const int per = TOKEN_WARPS / ks * wr;
    const dim3 grid((p.cols + per - 1) / per), block(TOKEN_THREADS);
    const size_t smem = static_cast<size_t>(chunks) * 16 * R;
    if (wr == 4) return launch_pdl(token_kernel<T, R, 4>, grid, block, smem, s, p, ks);
    if (wr == 2) return launch_pdl(token_kernel<T, R, 2>, grid, block, smem, s, p, ks);
    return launch_pdl(token_kernel<T, R, 1>, grid, block, smem, s, p, ks);
}
template <typename T>
cudaError_t pick_tokens(const TokenParams& p, cudaStream_t s) {
    return p.rows == 1 ? run_tokens<T, 1>(p, s) : run_tokens<T, 2>(p, s);
}

int blocks_for(long long items) {
    const long long b = (items + 255) / 256;
    return static_cast<int>(b < 1 ? 1 : b < 152 * 16 ? b : 152 * 16);
}

}  // namespace

cudaError_t linear_prepare() {
    cudaError_t e;
#define ANVIL_SMEM(kernel, bytes) \
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))) return e
    ANVIL_SMEM((pair_gemm_kernel<__nv_bfloat16, 64>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<__nv_bfloat16, 128>), Staging<128>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<__half, 64>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<__half, 128>), Staging<128>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<float, 64>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<float, 128>), Staging<128>::SMEM);
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 16>), RowShape<16>::smem(RowShape<16>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 32>), RowShape<32>::smem(RowShape<32>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 64>), RowShape<64>::smem(RowShape<64>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 128>), RowShape<128>::smem(RowShape<128>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 16>), RowShape<16>::smem(RowShape<16>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 32>), RowShape<32>::smem(RowShape<32>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 64>), RowShape<64>::smem(RowShape<64>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 128>), RowShape<128>::smem(RowShape<128>::STAGES));
#undef ANVIL_SMEM
    return cudaSuccess;
}

namespace {
template <typename T>
cudaError_t pick_pair(const PairGemmParams& p, int sm_count, cudaStream_t s) {
    return p.box_bytes == 64 ? run_pair<T, 64>(p, sm_count, s) : run_pair<T, 128>(p, sm_count, s);
}
}  // namespace

cudaError_t launch_pair_gemm(const PairGemmParams& p, int sm_count, cudaStream_t s) {
    if (p.epi.out_f32) return pick_pair<float>(p, sm_count, s);
    return p.f16 ? pick_pair<__half>(p, sm_count, s) : pick_pair<__nv_bfloat16>(p, sm_count, s);
}

cudaError_t launch_finish(const FinishParams& p, cudaStream_t s) {
    const int bias = p.bias.out ? (p.bias.cols + CS_COLS - 1) / CS_COLS : 0;
    const dim3 grid((p.tail[0].tiles + p.tail[1].tiles) * TAIL_BLOCKS + bias);
    if (p.f16) return launch_pdl(finish_kernel<__half>, grid, dim3(FINISH_THREADS), 0, s, p);
    return launch_pdl(finish_kernel<__nv_bfloat16>, grid, dim3(FINISH_THREADS), 0, s, p);
}

cudaError_t launch_tokens(const TokenParams& p, cudaStream_t s) {
    return p.f16 ? pick_tokens<__half>(p, s) : pick_tokens<__nv_bfloat16>(p, s);
}

cudaError_t launch_row_gemm(const RowGemmParams& p, int bn, int sm_count, cudaStream_t s) {
    switch (bn) {
        case 16: return p.f16 ? run_row<__half, 16>(p, sm_count, s) : run_row<__nv_bfloat16, 16>(p, sm_count, s);
        case 32: return p.f16 ? run_row<__half, 32>(p, sm_count, s) : run_row<__nv_bfloat16, 32>(p, sm_count, s);
        case 64: return p.f16 ? run_row<__half, 64>(p, sm_count, s) : run_row<__nv_bfloat16, 64>(p, sm_count, s);
        default: return p.f16 ? run_row<__half, 128>(p, sm_count, s) : run_row<__nv_bfloat16, 128>(p, sm_count, s);
    }
}

cudaError_t launch_repack(const RepackParams& p, cudaStream_t s) {
    long long most = 0;
    for (int j = 0; j < p.jobs; ++j) {
        const long long n = (p.job[j].cols + 7) / 8 * p.job[j].rows;
        if (n > most) most = n;
    }
    return launch_pdl(repack_kernel, dim3(blocks_for(most), p.jobs), dim3(256), 0, s, p);
}

namespace {
template <typename T>
cudaError_t run_act_grad(const ActGradParams& p, cudaStream_t s) {
    auto ok = [](const void* q, long long ld) { return !(reinterpret_cast<uintptr_t>(q) & 15) && ld % 8 == 0; };
    const bool vec = p.cols % 8 == 0 && ok(p.dy, p.lddy) && ok(p.z, p.z ? p.ldz : 0);
    const dim3 grid((p.cols + ACT_GRAD_COLS - 1) / ACT_GRAD_COLS, p.blocks_r), block(32 * AG_LANES);
#define ANVIL_ACT_CASE(A)                                                             \
    case A:                                                                           \
        return vec ? launch_pdl(act_grad_kernel<T, A, true>, grid, block, 0, s, p)    \
                   : launch_pdl(act_grad_kernel<T, A, false>, grid, block, 0, s, p)
    switch (p.act) {
        ANVIL_ACT_CASE(ACT_RELU);
        ANVIL_ACT_CASE(ACT_RELU2);
        ANVIL_ACT_CASE(ACT_GELU);
        ANVIL_ACT_CASE(ACT_GELU_TANH);
        ANVIL_ACT_CASE(ACT_SILU);
        default: break;
    }
    return vec ? launch_pdl(act_grad_kernel<T, ACT_NONE, true>, grid, block, 0, s, p)
               : launch_pdl(act_grad_kernel<T, ACT_NONE, false>, grid, block, 0, s, p);
#undef ANVIL_ACT_CASE
}
}  // namespace

cudaError_t launch_act_grad(const ActGradParams& p, cudaStream_t s) {
    return p.f16 ? run_act_grad<__half>(p, s) : run_act_grad<__nv_bfloat16>(p, s);
}

}  // namespace anvil
