// anvil_gated.cu -- the gated layer y = act(x G^T) * (x U^T), both products, the activation and the
// product in one kernel, and the elementwise part of its gradient.
//
//   forward   g = x G^T, u = x U^T, y = act(g) u               (g and u kept for the backward pass)
//   backward  dg = dy u act'(g), du = dy act(g)                (gated_grad_kernel)
//             dx = dg G + du U, dG = dg^T x, dU = du^T x       (anvil_multi.cu: one launch for the sum,
//                                                               one for both weights' gradients)
//
// Forward, many rows: the pair kernel (anvil_linear.cuh) as it is, but its two CTAs load their halves
// of operand B from different weights, rank 0 from G and rank 1 from U.  A tile's accumulator then
// holds g in its columns 0 to 127 and u in 128 to 255, each CTA has both for its 128 rows, and the
// epilogue multiplies registers with registers: g and u never leave the SM unless they are kept.  The
// products bound it, as they do the linear layer; the epilogue reads two columns and stores one (16384 x
// 8192 x 4096 bf16 1143 us, 1.92 PFLOP/s; 8192 x 2816 x 768 48 us, 54 with g and u kept; 1 x 2816 x 768 2.8).
// Few rows: the row kernel with 64 rows of either weight as the MMA's 128, joined through shared
// memory, where g and u of an element meet.  One or two tokens of small weights: the token kernel, a
// warp taking the same row of both.
#include <cuda_runtime.h>
#include <stdint.h>

#include "anvil_linear.cuh"

namespace anvil {

namespace {

constexpr int GROUP_COLS = GATED_COLS / EPI_GROUPS;  // 32 columns of y per epilogue group: a 64-byte box row

struct GatedPair {
    using Params = PairGatedParams;
    static constexpr bool MULTI = false, OWN = true, RANK_B = true, ONE_CHAIN = false;
    static constexpr int CHAIN = 0;
    struct Row {};
    static __device__ __forceinline__ Row load(const Params&, const Unit&, int) { return {}; }
    // tacc: this warp's lanes, column 0 of the accumulator
    template <typename T, int W>
    static __device__ __forceinline__ void tile(const Params& p, EpiState& x, uint32_t tacc, uint32_t tempty, const Unit& t,
                                                int row0, Row) {
        static_assert(W == 2 * GROUP_COLS, "a group's columns fill a box row");
        const GemmEpilogue& e = p.epi;
        const int col0 = t.tc * GATED_COLS + x.grp * GROUP_COLS;
        const uint32_t tg = tacc + x.grp * GROUP_COLS, tu = tg + GATED_COLS;
#pragma unroll 1
        for (int step = 0; step < 3; ++step) {  // g and u where they are kept, then y
            if ((step == 0 && !e.z) || (step == 1 && !p.z2)) continue;
            box_free(x);
#pragma unroll
            for (int c = 0; c < GROUP_COLS / 16; ++c) {
                float v[16];
                tmem_ld_16((step == 1 ? tu : tg) + c * 16, v);
                if (step == 2) {
                    float u[16];
                    tmem_ld_16(tu + c * 16, u);
                    act_values<16>(e.act, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] *= u[i];
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) sts128(Staging<W>::addr(x.box, x.r, c * 2 + j), Elem<T>::pack(v + 8 * j));
            }
            if (step == 2) release_acc(x, tempty);
            if (step == 0) send_box<uint16_t, W, false>(x, &p.tm_z, p.z_tma, e.z, e.ldz, row0, col0, p.rows, p.cols);
            else if (step == 1) send_box<uint16_t, W, false>(x, &p.tm_z2, p.z2_tma, p.z2, p.ldz2, row0, col0, p.rows, p.cols);
            else send_box<uint16_t, W, false>(x, &p.tm_out, p.out_tma, e.out, e.ldout, row0, col0, p.rows, p.cols);
        }
    }
};

// The tail tiles' parts: a block takes 16 rows of a tile, a thread one column of eight of them.
constexpr int GF_THREADS = 2 * GATED_COLS, GF_ROWS = 16, GF_BLOCKS = PAIR_ROWS / GF_ROWS;
template <typename T>
__global__ void __launch_bounds__(GF_THREADS) gated_finish_kernel(const __grid_constant__ GatedTailParams p) {
    pdl_allow_next();
    constexpr int N = GF_ROWS / 2;
    const int tile = blockIdx.x / GF_BLOCKS, r0 = blockIdx.x % GF_BLOCKS * GF_ROWS + threadIdx.x / GATED_COLS * N;
    const int c = threadIdx.x % GATED_COLS;
    int tr, tc;
    tile_at(p.split.whole + tile, p.tiles_r, p.tiles_c, &tr, &tc);
    const int col = tc * GATED_COLS + c, rows = p.rows - tr * PAIR_ROWS - r0;
    if (rows <= 0 || col >= p.cols) return;
    pdl_wait_previous();
    const bool first = tile < p.split.tiles_a;
    const int splits = first ? p.split.sa : p.split.sb;
    const int part0 = first ? tile * splits : p.split.tiles_a * p.split.sa + (tile - p.split.tiles_a) * splits;
    const float* part = p.part + (static_cast<size_t>(part0) * PAIR_ROWS + r0) * PAIR_COLS + c;
    float g[N], u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        g[i] = i < rows ? __ldcs(part + i * PAIR_COLS) : 0.f;
        u[i] = i < rows ? __ldcs(part + i * PAIR_COLS + GATED_COLS) : 0.f;
    }
    for (int s = 1; s < splits; ++s) {
        part += static_cast<size_t>(PAIR_ROWS) * PAIR_COLS;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < rows) {
                g[i] += __ldcs(part + i * PAIR_COLS);
                u[i] += __ldcs(part + i * PAIR_COLS + GATED_COLS);
            }
    }
    finish_gated<T, N>(p, g, u, static_cast<long long>(tr) * PAIR_ROWS + r0, rows, col);
}

// dg and du, eight columns a thread; both are operands and rounded to their type, as the linear
// layer's dz is, or kept in two parts.  Three reads and two writes of 2 bytes an element: HBM.
constexpr int GG_THREADS = 256, GG_UNROLL = 2;
template <typename T, int ACT, bool VEC>
__global__ void __launch_bounds__(GG_THREADS) gated_grad_kernel(const GatedGradParams p) {
    const T* dy = static_cast<const T*>(p.dy);
    const T* g = static_cast<const T*>(p.g);
    const T* u = static_cast<const T*>(p.u);
    T* dz = static_cast<T*>(p.dz);
    const long long part = p.rows * p.ldd;
    const int chunks = (p.cols + 7) / 8;
    pdl_allow_next();
    pdl_wait_previous();
    auto fetch = [&](const T* q, int c) {
        if constexpr (VEC) {
            return ldg_stream(q + c);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = c + e < p.cols ? __ldcs(reinterpret_cast<const uint16_t*>(q) + c + e) : 0u;
            return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
    };
    auto send = [&](const float (&v)[8], T* to) {
        const uint4 w = Elem<T>::pack(v);
        *reinterpret_cast<uint4*>(to) = w;
        if (p.two_parts) {
            float h[8];
            Elem<T>::unpack(w, h);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = isfinite(h[e]) ? v[e] - h[e] : 0.f;
            *reinterpret_cast<uint4*>(to + part) = Elem<T>::pack(h);
        }
    };
    Walk w(chunks, blockIdx.x * GG_THREADS + threadIdx.x, gridDim.x * GG_THREADS);
    while (w.row < p.rows) {
        uint4 wd[GG_UNROLL], wg[GG_UNROLL], wu[GG_UNROLL];
        long long row[GG_UNROLL];
        int c[GG_UNROLL];
#pragma unroll
        for (int k = 0; k < GG_UNROLL; ++k) {
            row[k] = w.row;
            c[k] = w.chunk * 8;
            w.next(chunks);
            if (row[k] >= p.rows) continue;
            wd[k] = fetch(dy + row[k] * p.lddy, c[k]);
            wg[k] = fetch(g + row[k] * p.ldg, c[k]);
            wu[k] = fetch(u + row[k] * p.ldu, c[k]);
        }
#pragma unroll
        for (int k = 0; k < GG_UNROLL; ++k) {
            if (row[k] >= p.rows) break;
            float d[8], a[8], b[8], dg[8];
            Elem<T>::unpack(wd[k], d);
            Elem<T>::unpack(wg[k], a);
            Elem<T>::unpack(wu[k], b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dg[e] = d[e] * b[e] * act_slope<ACT>(a[e]);
                d[e] *= act_value<ACT>(a[e]);
            }
            T* to = dz + row[k] * p.ldd + c[k];
            send(dg, to);
            send(d, to + (p.two_parts ? 2 : 1) * part);
        }
    }
}

template <typename T>
cudaError_t run_gated_grad(const GatedGradParams& p, cudaStream_t s) {
    auto ok = [](const void* q, long long ld) { return !(reinterpret_cast<uintptr_t>(q) & 15) && ld % 8 == 0; };
    const bool vec = p.cols % 8 == 0 && ok(p.dy, p.lddy) && ok(p.g, p.ldg) && ok(p.u, p.ldu);
    const long long items = (p.cols + 7) / 8 * p.rows, most = 152 * 16;
    long long blocks = (items + GG_THREADS * GG_UNROLL - 1) / (GG_THREADS * GG_UNROLL);
    if (blocks > most) blocks = most;
    const dim3 grid(static_cast<unsigned>(blocks)), block(GG_THREADS);
#define ANVIL_ACT_CASE(A)                                                            \
    case A:                                                                          \
        return vec ? launch_pdl(gated_grad_kernel<T, A, true>, grid, block, 0, s, p) \
                   : launch_pdl(gated_grad_kernel<T, A, false>, grid, block, 0, s, p)
    switch (p.act) {
        ANVIL_ACT_CASE(ACT_RELU);
        ANVIL_ACT_CASE(ACT_RELU2);
        ANVIL_ACT_CASE(ACT_GELU);
        ANVIL_ACT_CASE(ACT_GELU_TANH);
        ANVIL_ACT_CASE(ACT_SILU);
        default: break;
    }
    return vec ? launch_pdl(gated_grad_kernel<T, ACT_NONE, true>, grid, block, 0, s, p)
               : launch_pdl(gated_grad_kernel<T, ACT_NONE, false>, grid, block, 0, s, p);
#undef ANVIL_ACT_CASE
}

}  // namespace

cudaError_t gated_prepare() {
    cudaError_t e;
#define ANVIL_SMEM(kernel, bytes) \
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))) return e
#define ANVIL_ROWS(T, BN) ANVIL_SMEM((row_gemm_kernel<T, BN, GatedRows>), RowShape<BN>::smem(RowShape<BN>::STAGES))
    ANVIL_SMEM((pair_gemm_kernel<__nv_bfloat16, 64, GatedPair>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<__half, 64, GatedPair>), Staging<64>::SMEM);
    ANVIL_ROWS(__nv_bfloat16, 16);
    ANVIL_ROWS(__nv_bfloat16, 32);
    ANVIL_ROWS(__half, 16);
    ANVIL_ROWS(__half, 32);
#undef ANVIL_ROWS
#undef ANVIL_SMEM
    return cudaSuccess;
}

cudaError_t launch_pair_gated(const PairGatedParams& p, int sm_count, cudaStream_t s) {
    return p.f16 ? run_pair<__half, 64, GatedPair>(p, sm_count, s) : run_pair<__nv_bfloat16, 64, GatedPair>(p, sm_count, s);
}

namespace {
template <typename T>
cudaError_t pick_row(const RowGatedParams& p, int bn, int sm_count, cudaStream_t s) {
    return bn == 16 ? run_row<T, 16, GatedRows>(p, sm_count, s) : run_row<T, 32, GatedRows>(p, sm_count, s);
}
}  // namespace

cudaError_t launch_row_gated(const RowGatedParams& p, int bn, int sm_count, cudaStream_t s) {
    return p.f16 ? pick_row<__half>(p, bn, sm_count, s) : pick_row<__nv_bfloat16>(p, bn, sm_count, s);
}

cudaError_t launch_tokens_gated(const TokenGatedParams& p, cudaStream_t s) {
    return p.f16 ? pick_tokens<__half, GatedTokens>(p, s) : pick_tokens<__nv_bfloat16, GatedTokens>(p, s);
}

cudaError_t launch_gated_finish(const GatedTailParams& p, cudaStream_t s) {
    const dim3 grid(p.tiles * GF_BLOCKS), block(GF_THREADS);
    return p.f16 ? launch_pdl(gated_finish_kernel<__half>, grid, block, 0, s, p)
                 : launch_pdl(gated_finish_kernel<__nv_bfloat16>, grid, block, 0, s, p);
}

cudaError_t launch_gated_grad(const GatedGradParams& p, cudaStream_t s) {
    return p.f16 ? run_gated_grad<__half>(p, s) : run_gated_grad<__nv_bfloat16>(p, s);
}

}  // namespace anvil
