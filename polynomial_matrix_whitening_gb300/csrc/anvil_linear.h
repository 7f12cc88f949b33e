// anvil_linear.h -- parameter blocks and launchers of the linear layer's kernels (internal
// to libanvil).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace anvil {

// activation codes of include/anvil.h (anvil_activation)
enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_SILU = 5, ACT_COUNT = 6 };

// What follows a product's fp32 accumulator v at (row, col):
//   v += bias[col];  z = v (stored if z);  v = act(v);  v += in;  out = v
struct GemmEpilogue {
    const void* bias;     // [cols] or null
    const void* in;       // residual (16 bit) or the gradient so far (out's type), or null
    void* z;              // or null
    void* out;
    long long ldin, ldz, ldout;
    int bias_f32;         // bias is fp32 (else the operands' type)
    int act;
    int out_f32;          // out (and in) are fp32
    const float* scale;   // null, or what v is multiplied by first (PairMultiParams only)
};

// Which tiles are computed in one piece and which in parts.  The first `whole` tiles are
// whole.  The others (the tail) are split along k, the first `tiles_a` of them into `sa` parts
// of `kba` 64-deep k-blocks, the rest into `sb` of `kbb`; the fp32 parts go to scratch, a
// 256 x 256 block each, in that order.  Of `pairs` CTA pairs the first `early` take the parts
// of the first kind, the others those of the second.
struct TileSplit {
    int whole, pairs, early, tiles_a, sa, kba, sb, kbb;
};

// C [rows, cols] = sum_k A[row, k] B[col, k].  An operand is K-major (stored [row][k]) or
// MN-major (stored [k][row]).
struct PairGemmParams {
    CUtensorMap tm_a, tm_b, tm_in, tm_out, tm_z, tm_part;
    GemmEpilogue epi;
    int rows, cols, k;
    int a_mn, b_mn;
    int f16;                        // operands are fp16 (else bf16)
    int in_tma, out_tma, z_tma;     // through tensor maps (16-byte aligned rows)
    int box_bytes;                  // row of a staging box: 64 (six stages) or 128 (five)
    int tiles_r, tiles_c;           // 256 x 256 output tiles
    TileSplit split;
    int units;                      // of work: whole tiles and the turns of the tail (unit_of)
    int one_chain;                  // the fp32 result is one chain of products
    int overlap_next;               // the next kernel may start before this one has ended
    int overlap_previous;           // and this one before the previous one has (both products of a backward pass)
    unsigned* err;
};
// Several products in one launch.  A result's contraction may be in up to four segments, each with
// operands of its own (a sum of products); and there may be two results of the same sizes, the second
// one's rows of tiles after the first one's (tiles_r counts both, rows one).
struct PairMultiParams : PairGemmParams {
    CUtensorMap tm_a2[3], tm_b2[3];  // operands of number 1 to 3: result * segments + segment (0: tm_a, tm_b)
    CUtensorMap tm_in2, tm_out2;     // the second result's
    GemmEpilogue epi2;
    int result_tiles;                // rows of tiles of one result
    int segments, seg_kb;            // k-blocks of a segment
};
// What is added up after the products, in one launch: the tail tiles' parts of up to two
// products, with what follows the accumulator, and the column sums of a bias gradient.
struct TailSumParams {
    GemmEpilogue epi;
    const float* part;
    int rows, cols, tiles_r, tiles_c, tiles;  // tiles: of the tail (0: nothing to do)
    TileSplit split;
    GemmEpilogue epi2;      // of a second result,
    int result_tiles;       // whose rows of tiles come after these (0: there is none)
};
struct ColumnSumParams {
    const float* part;  // [blocks][cols]
    float* out;         // (+)= the sum over the blocks, in order (null: nothing to do)
    int blocks, cols, accumulate;
};
struct FinishParams {
    TailSumParams tail[2];
    ColumnSumParams bias;
    int f16;            // 16-bit results are fp16 (else bf16)
};
// A = the operand whose rows run along the output's contiguous dimension ("cols" above),
// B = the few rows: out[b][a].
struct RowGemmParams {
    CUtensorMap tm_a, tm_b;
    GemmEpilogue epi;               // columns are A's rows, rows are B's rows
    int na, nb, k;                  // A's rows, B's rows, contraction
    int a_mn;                       // A MN-major (B is always K-major)
    int f16;
    int splits;                     // cluster size along k
    int stages;                     // of the ring (set by the launcher)
    int kb_per_split;
    unsigned* err;
};

// One or two rows (tokens) and a weight stored [cols][k], both on 16-byte rows.
struct TokenParams {
    const void* x;
    const void* w;
    GemmEpilogue epi;
    long long ldx, ldw;
    int rows, cols, k;
    int f16;
};
// The gated layer: y = act(g) u with g = x G^T, u = x U^T, n columns each.  A tile of the pair kernel
// is 256 rows by 128 columns of both (p.cols is n; tm_b is G's map, tm_b2 U's; g goes to epi.z, u to z2
// where they are kept); the row kernel's 128 weight rows are 64 of each.
struct PairGatedParams : PairGemmParams {
    CUtensorMap tm_b2, tm_z2;
    void* z2;
    long long ldz2;
    int z2_tma;
};
struct RowGatedParams : RowGemmParams {
    CUtensorMap tm_a2;
    void* z2;
    long long ldz2;
};
struct TokenGatedParams : TokenParams {
    const void* w2;
    long long ldw2;
    void* z2;
    long long ldz2;
};
// The tail tiles' parts of a gated product.
struct GatedTailParams {
    GemmEpilogue epi;
    void* z2;
    long long ldz2;
    const float* part;
    int rows, cols, tiles_r, tiles_c, tiles, f16;
    TileSplit split;
};
constexpr int GATED_COLS = 128;  // of y in a tile
constexpr int TOKEN_ROWS = 2;
constexpr int TOKEN_CHUNKS = 3008;  // 16-byte chunks of the tokens that shared memory takes (47 KB, 48 with what is static)

constexpr int GEMM_BK = 64;    // k-block: one 128-byte swizzle row of 16-bit elements
constexpr int PAIR_ROWS = 256; // output rows and columns of a CTA pair's tile
constexpr int PAIR_COLS = 256;
constexpr int ROW_TILE_A = 128;    // weight rows of a row kernel's block
constexpr int ROW_TWO_TOKENS = 32; // tokens of a block up to which two share an SM

cudaError_t linear_prepare();
cudaError_t launch_pair_gemm(const PairGemmParams& p, int sm_count, cudaStream_t stream);
cudaError_t gated_prepare();
cudaError_t launch_pair_gated(const PairGatedParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_row_gated(const RowGatedParams& p, int bn, int sm_count, cudaStream_t stream);
cudaError_t launch_tokens_gated(const TokenGatedParams& p, cudaStream_t stream);
cudaError_t launch_gated_finish(const GatedTailParams& p, cudaStream_t stream);
// dg = dy u act'(g) and du = dy act(g), rounded to the operands' type, [rows, ldd] each; two parts:
// what the rounding drops, rounded itself, behind each (dg, its rest, du, its rest).
struct GatedGradParams {
    const void* dy;
    const void* g;
    const void* u;
    void* dz;
    int two_parts;
    long long rows, lddy, ldg, ldu, ldd;
    int cols, act, f16;
};
cudaError_t launch_gated_grad(const GatedGradParams& p, cudaStream_t stream);
// The head: z = x W^T by tiles that are used and dropped (p.cols columns from column `first` of the vocabulary).
// Statistics: of each row's 64 columns (m, S), the largest z and S = sum_j e^(z_j - m), and the target's z.
// Gradient: out = g (e^(z - lse) - [j = target]) (times *scale), 16 bit.
struct PairHeadParams : PairGemmParams {
    const void* targets;
    int target64;
    int first;
    float2* stats;        // [4 tiles_c][rows]
    float* hit;           // [rows]
    const float* lse;     // [rows]
    const float* grad;    // [rows]
    const float* scale;
};
constexpr int HEAD_STATS_COLS = 64;  // columns behind one pair of statistics
constexpr int HEAD_CHAIN_KB = 16;    // k-blocks of a chain of the logits behind loss and lse
// The same for few rows: statistics [blocks of 128 columns][rows].
struct RowHeadParams : RowGemmParams {
    const void* targets;
    int target64;
    float2* stats;
    float* hit;
};
// One or two rows, the weight [cols][k] on 16-byte rows: statistics [blocks][rows].
struct TokenHeadParams {
    const void* x;
    const void* w;
    long long ldx, ldw;
    int rows, cols, k, f16;
    const void* targets;
    int target64;
    float2* stats;
    float* hit;
};
constexpr int HEAD_TOKENS = 2, HEAD_TOKEN_VALUES = 16384;  // rows; values of x, fp32 in shared memory
constexpr int HEAD_TOKEN_GROUP = 4, HEAD_TOKEN_WARPS = 8;  // weight rows of a warp at a time, warps of a block
// Blocks: two for each of a GB300's SMs, as far as there are groups of weight rows for their warps.
inline int head_token_blocks(int cols) {
    const int per = HEAD_TOKEN_GROUP * HEAD_TOKEN_WARPS, all = (cols + per - 1) / per;
    return all < 152 * 2 ? all : 152 * 2;
}
struct HeadJoinParams {
    const float2* stats;
    const float* hit;
    const void* targets;
    float* loss;          // or null
    float* lse;           // or null
    long long rows;
    int parts, vocab, target64;
};
// scale[1] = the largest finite |grad| of rows that count (fp16: over 2^13), scale[0] = 1 / scale[1]
struct HeadScaleParams {
    const float* grad;
    const void* targets;
    float* scale;
    long long rows;
    int target64, f16;
};
// dst [rows, cols] 16 bit = src fp32 [rows, cols] (times *scale)
struct HeadRoundParams {
    const float* src;
    void* dst;
    const float* scale;
    long long rows, ldd;
    int cols, f16;
};
cudaError_t head_prepare();
cudaError_t launch_head_stats(const PairHeadParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_head_tokens(const TokenHeadParams& p, cudaStream_t stream);
// bn: rows of x per block (16 or 32)
cudaError_t launch_head_rows(const RowHeadParams& p, int bn, int sm_count, cudaStream_t stream);
cudaError_t launch_head_join(const HeadJoinParams& p, cudaStream_t stream);
cudaError_t launch_head_dlogits(const PairHeadParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_head_scale(const HeadScaleParams& p, cudaStream_t stream);
cudaError_t launch_head_round(const HeadRoundParams& p, cudaStream_t stream);
cudaError_t multi_prepare();
cudaError_t launch_pair_multi(const PairMultiParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_finish(const FinishParams& p, cudaStream_t stream);
cudaError_t launch_tokens(const TokenParams& p, cudaStream_t stream);
// bn: B's rows per block (16, 32, 64 or 128)
cudaError_t launch_row_gemm(const RowGemmParams& p, int bn, int sm_count, cudaStream_t stream);

// dst (`rows` rows of `cols` elements, rounded up to eights, row stride ldd, ldd % 8 == 0) <- src
// (src_rows rows, row stride lds), zeros beyond; 16-bit elements, for up to four arrays.
struct Repack {
    const uint16_t* src;
    uint16_t* dst;
    long long rows, src_rows, lds, ldd;
    int cols;
};
struct RepackParams {
    Repack job[4];
    int jobs;
};
cudaError_t launch_repack(const RepackParams& p, cudaStream_t stream);

// dz = dy * act'(z) (rounded to the operands' type for the products; may be null) and the
// column sums of the unrounded dz (partial rows; may be null).  Two parts: what the rounding
// drops, rounded itself, in the second half of dz's rows.
struct ActGradParams {
    const void* dy;
    const void* z;       // null: dz = dy
    void* dz;            // [rows, ldd] or null
    int two_parts;
    float* part;         // [blocks_r][cols] or null
    long long rows, lddy, ldz, ldd;
    int cols, act, f16;
    int rows_per_block, blocks_r;
};
constexpr int ACT_GRAD_COLS = 256;  // columns per block
constexpr int ACT_GRAD_BLOCKS = 3;  // blocks that an SM holds
cudaError_t launch_act_grad(const ActGradParams& p, cudaStream_t stream);

}  // namespace anvil
