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
#include <stdint.h>

#include "anvil_linear.cuh"

namespace anvil {

namespace {

// The tail tiles of pair_gemm_kernel: the parts of each element, in order, then what follows
// the accumulator.  A block takes 16 rows of a tile, a thread one column of them, so that
// neighbouring lanes are neighbouring elements whatever the arrays' alignment.
constexpr int FINISH_THREADS = PAIR_COLS;
constexpr int TAIL_ROWS = 16, TAIL_BLOCKS = PAIR_ROWS / TAIL_ROWS;
// MULTI: of a launch of several products (a second result, scaled results); apart, since a choice of
// parameters by a value costs the others 2 us (1000 x 2815 x 771).
template <typename T, bool MULTI>
__device__ __forceinline__ void tail_sum(const TailSumParams& p, int block) {
    const int tile = block / TAIL_BLOCKS, r0 = block % TAIL_BLOCKS * TAIL_ROWS;
    int tr, tc;
    tile_at(p.split.whole + tile, p.tiles_r, p.tiles_c, &tr, &tc);
    bool second = false;
    if constexpr (MULTI) second = p.result_tiles && tr >= p.result_tiles;
    if (second) tr -= p.result_tiles;
    const GemmEpilogue& e = second ? p.epi2 : p.epi;
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
    if constexpr (MULTI) {
        // in order, four parts on their way at a time (one after the other, 64 parts of a few rows took 14 us)
        constexpr size_t PART = static_cast<size_t>(PAIR_ROWS) * PAIR_COLS;
        part += PART;
        for (int s = 1; s < splits; s += 4, part += 4 * PART) {
            float t[4][TAIL_ROWS];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < TAIL_ROWS; ++i) t[k][i] = s + k < splits && i < rows ? __ldcs(part + k * PART + i * PAIR_COLS) : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < TAIL_ROWS; ++i)
                    if (s + k < splits) v[i] += t[k][i];
        }
    } else {
        for (int s = 1; s < splits; ++s) {
            part += static_cast<size_t>(PAIR_ROWS) * PAIR_COLS;
#pragma unroll
            for (int i = 0; i < TAIL_ROWS; ++i) v[i] += __ldcs(part + i * PAIR_COLS);
        }
    }
    if (MULTI && e.scale) {
        const float scale = *e.scale;
#pragma unroll
        for (int i = 0; i < TAIL_ROWS; ++i) v[i] *= scale;
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
template <typename T, bool MULTI>
__global__ void __launch_bounds__(FINISH_THREADS) finish_kernel(const __grid_constant__ FinishParams p) {
    pdl_allow_next();
    int b = blockIdx.x;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const TailSumParams& t = p.tail[j];
        const int blocks = t.tiles * TAIL_BLOCKS;
        if (b < blocks) {
            if (t.epi.out_f32) tail_sum<float, MULTI>(t, b);
            else tail_sum<T, MULTI>(t, b);
            return;
        }
        b -= blocks;
    }
    column_sum(p.bias, b);
}

// ---------------------------------------------------------------- around the products
// Eight columns per thread; the last chunk of a row may be partial.
__global__ void __launch_bounds__(256) repack_kernel(const __grid_constant__ RepackParams q) {
    const Repack& p = q.job[blockIdx.y];
    pdl_wait_previous();  // (the product starts after this kernel: its shared memory would take the L1 that the loads need)
    const int chunks = (p.cols + 7) / 8;
    for (Walk at(chunks, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256); at.row < p.rows; at.next(chunks)) {
        const long long row = at.row;
        const int c = at.chunk * 8;
        const uint16_t* s = p.src + row * p.lds + c;
        uint4 to;
        if (row < p.src_rows && c + 8 <= p.cols) {
            // words, of which an odd start is half a word off
            uint32_t w[5];
            const bool odd = (reinterpret_cast<uintptr_t>(s) & 2) != 0;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(s + odd);
            w[0] = odd ? *s : 0u;
#pragma unroll
            for (int e = 0; e < 3; ++e) w[e + 1] = q[e];
            w[4] = odd ? s[7] : q[3];
            to = odd ? make_uint4(w[0] | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16 | w[4] << 16)
                     : make_uint4(w[1], w[2], w[3], w[4]);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = c + e < p.cols && row < p.src_rows ? s[e] : 0u;
            to = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
        *reinterpret_cast<uint4*>(p.dst + row * p.ldd + c) = to;
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

int blocks_for(long long items) {
    const long long b = (items + 255) / 256;
    return static_cast<int>(b < 1 ? 1 : b < 152 * 16 ? b : 152 * 16);
}

}  // namespace

cudaError_t linear_prepare() {
    cudaError_t e;
#define ANVIL_SMEM(kernel, bytes) \
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))) return e
    ANVIL_SMEM((pair_gemm_kernel<__nv_bfloat16, 64, PlainPair>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<__nv_bfloat16, 128, PlainPair>), Staging<128>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<__half, 64, PlainPair>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<__half, 128, PlainPair>), Staging<128>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<float, 64, PlainPair>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<float, 128, PlainPair>), Staging<128>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<float, 64, SumPair>), Staging<64>::SMEM);
    ANVIL_SMEM((pair_gemm_kernel<float, 128, SumPair>), Staging<128>::SMEM);
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 16, PlainRows>), RowShape<16>::smem(RowShape<16>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 32, PlainRows>), RowShape<32>::smem(RowShape<32>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 64, PlainRows>), RowShape<64>::smem(RowShape<64>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__nv_bfloat16, 128, PlainRows>), RowShape<128>::smem(RowShape<128>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 16, PlainRows>), RowShape<16>::smem(RowShape<16>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 32, PlainRows>), RowShape<32>::smem(RowShape<32>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 64, PlainRows>), RowShape<64>::smem(RowShape<64>::STAGES));
    ANVIL_SMEM((row_gemm_kernel<__half, 128, PlainRows>), RowShape<128>::smem(RowShape<128>::STAGES));
#undef ANVIL_SMEM
    return cudaSuccess;
}

namespace {
template <typename T>
cudaError_t pick_pair(const PairGemmParams& p, int sm_count, cudaStream_t s) {
    return p.box_bytes == 64 ? run_pair<T, 64, PlainPair>(p, sm_count, s) : run_pair<T, 128, PlainPair>(p, sm_count, s);
}
}  // namespace

cudaError_t launch_pair_gemm(const PairGemmParams& p, int sm_count, cudaStream_t s) {
    if (p.one_chain) return p.box_bytes == 64 ? run_pair<float, 64, SumPair>(p, sm_count, s) : run_pair<float, 128, SumPair>(p, sm_count, s);
    if (p.epi.out_f32) return pick_pair<float>(p, sm_count, s);
    return p.f16 ? pick_pair<__half>(p, sm_count, s) : pick_pair<__nv_bfloat16>(p, sm_count, s);
}

cudaError_t launch_finish(const FinishParams& p, cudaStream_t s) {
    const int bias = p.bias.out ? (p.bias.cols + CS_COLS - 1) / CS_COLS : 0;
    const dim3 grid((p.tail[0].tiles + p.tail[1].tiles) * TAIL_BLOCKS + bias);
    const dim3 block(FINISH_THREADS);
    bool multi = false;
    for (const TailSumParams& t : p.tail) multi = multi || (t.tiles && (t.result_tiles || t.epi.scale));
    if (p.f16) return multi ? launch_pdl(finish_kernel<__half, true>, grid, block, 0, s, p) : launch_pdl(finish_kernel<__half, false>, grid, block, 0, s, p);
    return multi ? launch_pdl(finish_kernel<__nv_bfloat16, true>, grid, block, 0, s, p)
                 : launch_pdl(finish_kernel<__nv_bfloat16, false>, grid, block, 0, s, p);
}

cudaError_t launch_tokens(const TokenParams& p, cudaStream_t s) {
    return p.f16 ? pick_tokens<__half, PlainTokens>(p, s) : pick_tokens<__nv_bfloat16, PlainTokens>(p, s);
}

cudaError_t launch_row_gemm(const RowGemmParams& p, int bn, int sm_count, cudaStream_t s) {
    switch (bn) {
        case 16: return p.f16 ? run_row<__half, 16, PlainRows>(p, sm_count, s) : run_row<__nv_bfloat16, 16, PlainRows>(p, sm_count, s);
        case 32: return p.f16 ? run_row<__half, 32, PlainRows>(p, sm_count, s) : run_row<__nv_bfloat16, 32, PlainRows>(p, sm_count, s);
        case 64: return p.f16 ? run_row<__half, 64, PlainRows>(p, sm_count, s) : run_row<__nv_bfloat16, 64, PlainRows>(p, sm_count, s);
        default: return p.f16 ? run_row<__half, 128, PlainRows>(p, sm_count, s) : run_row<__nv_bfloat16, 128, PlainRows>(p, sm_count, s);
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
