// anvil_block_api.cu -- the C ABI of the operators around the banks (include/anvil.h):
// layer norm, the linear layer and token log probabilities.  Argument checks (before any
// CUDA call), workspace layouts, tensor maps, and the choice of kernel and tile shape from
// the sizes, types and alignment.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/anvil.h"
#include "anvil_host.h"
#include "anvil_linear.h"
#include "anvil_logprob.h"
#include "anvil_norm.h"

using namespace anvil;

static_assert(ANVIL_ACT_SILU == ACT_SILU && ANVIL_ACT_RELU2 == ACT_RELU2, "activation codes of include/anvil.h");
static_assert(ANVIL_MAX_TOP == LOGPROB_MAX_TOP, "ANVIL_MAX_TOP");
static_assert(ANVIL_DZ_TWO_PARTS >= ACT_COUNT, "a bit of its own beside the activation codes");

namespace {

int size_of(int dtype) { return dtype == ANVIL_F32 ? 4 : 2; }
bool valid_dtype(int dtype) { return dtype == ANVIL_F32 || dtype == ANVIL_BF16 || dtype == ANVIL_F16; }

// A row-major array of the call: `rows` rows of `width` bytes, `ld` bytes apart.
struct Area {
    uintptr_t p;
    int64_t rows, ld, width;
    bool written;
};

Area area(const void* p, int64_t rows, int64_t cols, int64_t ld, int es, bool written) {
    return {reinterpret_cast<uintptr_t>(p), rows, rows > 1 ? ld * es : cols * es, cols * es, written};
}

// Whether two areas share a byte.  Interleaved rows (the same row stride) share none when
// their columns are disjoint; other areas are taken as the whole range they span.
bool share(const Area& a, const Area& b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
    const Range ra = {a.p, a.p + static_cast<uintptr_t>((a.rows - 1) * a.ld + a.width)};
    const Range rb = {b.p, b.p + static_cast<uintptr_t>((b.rows - 1) * b.ld + b.width)};
    if (!overlap(ra, rb)) return false;
    if (a.rows > 1 && b.rows > 1 && a.ld == b.ld) {
        const int64_t off = b.p >= a.p ? static_cast<int64_t>((b.p - a.p) % static_cast<uintptr_t>(a.ld))
                                       : (a.ld - static_cast<int64_t>((a.p - b.p) % static_cast<uintptr_t>(a.ld))) % a.ld;
        return !(off >= a.width && off + b.width <= a.ld);
    }
    return true;
}
bool same(const Area& a, const Area& b) { return a.p == b.p && a.rows == b.rows && a.ld == b.ld && a.width == b.width; }

// Every written area against every other; `inplace` lists the pairs (written, other) that
// may be the very same array.
anvil_status check_areas(const Area* a, int n, const int (*inplace)[2], int npairs) {
    for (int i = 0; i < n; ++i) {
        if (!a[i].written) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || (a[j].written && j < i) || !share(a[i], a[j])) continue;
            bool ok = false;
            for (int q = 0; q < npairs; ++q)
                ok = ok || (inplace[q][0] == i && inplace[q][1] == j && same(a[i], a[j]));
            if (!ok) return ANVIL_ERR_ALIAS;
        }
    }
    return ANVIL_OK;
}

bool misaligned(const void* p, int es) { return (reinterpret_cast<uintptr_t>(p) & (es - 1)) != 0; }
bool bad_ld(int64_t rows, int64_t cols, int64_t ld) { return rows > 1 && ld < cols; }

anvil_status check_workspace(const void* ws, size_t bytes, size_t need, const Area* a, int n) {
    if (need == 0) return ANVIL_OK;
    if (!ws || bytes < need) return ANVIL_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255) return ANVIL_ERR_ALIGNMENT;
    const Area w = {reinterpret_cast<uintptr_t>(ws), 1, static_cast<int64_t>(need), static_cast<int64_t>(need), true};
    for (int i = 0; i < n; ++i)
        if (share(w, a[i])) return ANVIL_ERR_ALIAS;
    return ANVIL_OK;
}

// ---------------------------------------------------------------- layer norm
anvil_status check_norm_sizes(int64_t rows, int width, int dtype, int weight_dtype) {
    if (rows < 0 || width < 1 || !valid_dtype(dtype)) return ANVIL_ERR_INVALID_ARG;
    if (weight_dtype != ANVIL_F32 && weight_dtype != dtype) return ANVIL_ERR_INVALID_ARG;
    if (rows > ANVIL_MAX_ROWS || width > ANVIL_MAX_WIDTH) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    return ANVIL_OK;
}

// The SM count the work is divided for (a GB300's; one constant, so that the workspaces need
// no device query and the order of the sums is the same everywhere).
constexpr int PLAN_SMS = 152;

size_t norm_bwd_bytes(const anvil_layernorm_grad_desc* d) {
    if (d->rows == 0 || (!d->dweight && !d->dbias)) return 0;
    const int blocks = norm_bwd_max_blocks(d->rows, d->width, d->dtype);
    return blocks > 1 ? align256(sizeof(float) * 2 * static_cast<size_t>(blocks) * d->width) : 0;
}

// ---------------------------------------------------------------- the linear layer
anvil_status check_linear_sizes(int64_t rows, int n, int k, int dtype, int act) {
    if (rows < 0 || n < 1 || k < 1 || (dtype != ANVIL_BF16 && dtype != ANVIL_F16) || act < 0 || act >= ACT_COUNT)
        return ANVIL_ERR_INVALID_ARG;
    if (rows > ANVIL_MAX_ROWS || n > ANVIL_MAX_FEATURES || k > ANVIL_MAX_FEATURES) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    // 32-bit tile numbers
    const int64_t t = (rows + 127) / 128;
    if (t * ((n + 127) / 128) >= (1ll << 30) || t * ((k + 127) / 128) >= (1ll << 30)) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    return ANVIL_OK;
}

// A 16-bit matrix operand as it is stored: `rows` rows of `cols` elements.
struct Stored {
    const void* p;
    int64_t rows, ld;
    int cols;
};

// Bytes of the 16-byte-aligned copy an operand needs (0: none).
size_t copy_bytes(const Stored& s) {
    if (aligned16(s.p, s.ld, 2, s.rows)) return 0;
    return align256(2 * static_cast<size_t>(s.rows) * ((s.cols + 7) & ~7));
}
Stored with_copy(const Stored& s, void* copy) {
    Stored r = s;
    r.p = copy;
    r.ld = (s.cols + 7) & ~7;
    return r;
}

// Tensor map of a row-major matrix [outer][inner], boxes of box1 rows by box0 elements
// (128 or 64 bytes, the swizzle of that size).  A third dimension of one, for the 3-D copies.
anvil_status encode(CUtensorMap* map, int es, bool f16, const void* base, int64_t inner, int64_t outer, int64_t ld, int box0,
                    int box1) {
    // a row stride is only used where there are several rows; keep it a multiple of 16 bytes
    const int64_t ldb = outer > 1 ? ld * es : (inner * es + 15) / 16 * 16;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer), 1};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ldb), static_cast<cuuint64_t>(ldb)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box0), static_cast<cuuint32_t>(box1), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType type = es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : f16   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = g_encode(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE,
                                box0 * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char text[64];
        snprintf(text, sizeof(text), "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
        set_error_text(text);
        return ANVIL_ERR_CUDA;
    }
    return ANVIL_OK;
}

// One product C [rows, cols] = A B^T over k, from operands on 16-byte rows: A as stored
// [rows][k] (or [k][rows] when a_mn), B as [cols][k] (or [k][cols] when b_mn).
struct Product {
    Stored a, b;
    bool a_mn, b_mn;
    int64_t rows;
    int cols;
    int64_t k;
    bool f16;
    GemmEpilogue epi;
    float* part;  // scratch of the tail tiles' parts
    bool overlap_next, overlap_previous;  // pair_gemm_kernel's flags
};

// How a product runs.
struct Plan {
    bool tokens;      // token_kernel
    bool few;         // row_gemm_kernel
    int bn;           // few: B rows of a block,
    int splits, kb;   //      parts of the contraction and the k-blocks of each
    TileSplit split;  // pair_gemm_kernel
    int tail, units;  // tiles in parts; units of work
    size_t part;      // bytes of the parts
    double cost;      // SM cycles, estimated
};

constexpr int FEW_ROWS = 256;  // row_gemm_kernel is considered up to here
constexpr int PLAN_PAIRS = PLAN_SMS / 2;

// What the pair kernel finds when it starts: of the grid's pairs the first `early` are free
// at once, the others `delay` SM cycles later (the last turn of the product before it).
struct Start {
    int early;
    double delay;
};
constexpr Start ALL_FREE = {PLAN_PAIRS, 0.0};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Blocks of 128 weight rows by 16 to 128 tokens, the contraction whole or split over a
// cluster.  Estimated times in SM cycles, from the kernel's own time stamps: 545 for a
// k-block (the MMA reads its 128-row operand at 32 bytes a cycle, whatever the tokens),
// 1700 to the first and from the last, 28 for a token's column; a join 2500, and 250 for
// a token's column of each block's share.
void plan_few(int64_t rows, int cols, int64_t kb, double epilogue, Plan* p) {
    for (int bn = 16; bn <= 128; bn *= 2) {
        const int64_t tiles = ceil_div(cols, ROW_TILE_A) * ceil_div(rows, bn);
        const double columns = static_cast<double>(bn < rows ? bn : rows) * (epilogue / 2500.0);
        for (int s = 1; s <= 8; s *= 2) {
            const int64_t per = ceil_div(kb, s);
            if (s > 1 && (per * (s - 1) >= kb || tiles * s > PLAN_SMS)) break;  // every split has work
            const double turns = static_cast<double>(ceil_div(tiles * s, PLAN_SMS));
            const double finish = s == 1 ? 28.0 * columns : 2500.0 + 10.0 * bn + 60.0 * columns / s;
            // (two blocks of up to 32 tokens share an SM: one's start and end beside the other's products)
            const double ends = turns > 1 && bn <= ROW_TWO_TOKENS ? 0.5 * turns : turns;
            const double cost = turns * per * 545.0 + ends * (1700.0 + finish);
            if (p->cost == 0 || cost < p->cost) {
                p->cost = cost;
                p->few = true;
                p->bn = bn;
                p->splits = s;
                p->kb = static_cast<int>(per);
            }
        }
    }
}

// Tiles in one piece, turn by turn of the grid's pairs; the tiles left over for a last turn
// that would not be full, or all of them, may go in parts instead (split along k, or whole
// but with the epilogue left to the finishing kernel).  Estimated times in SM cycles, fitted
// to measurements: 550 for a k-block, 2500 for filling the pipeline, 7500 for starting and
// leaving the kernel; an epilogue overlaps the next tile's products; parts cost 8000 for
// the finishing kernel and 200 a unit for their way through memory.
constexpr double KB_CYCLES = 550.0, FILL_CYCLES = 2500.0, LEAVE_CYCLES = 7500.0, FINISH_CYCLES = 8000.0, PART_CYCLES = 200.0;

int64_t tiles_of(int64_t rows, int cols) { return ceil_div(rows, PAIR_ROWS) * ceil_div(cols, PAIR_COLS); }
double turn_cycles(int64_t kb, double epilogue) { return kb * KB_CYCLES > epilogue ? kb * KB_CYCLES : epilogue; }

void set_whole(int64_t tiles, double cost, Plan* p) {
    memset(p, 0, sizeof(*p));
    p->cost = cost;
    p->split = {static_cast<int>(tiles), PLAN_PAIRS, PLAN_PAIRS, 0, 1, 0, 1, 0};
    p->units = static_cast<int>(tiles);
}

void plan_whole(int64_t tiles, int64_t kb, double epilogue, Start at, Plan* p) {
    const double products = kb * KB_CYCLES, turn = turn_cycles(kb, epilogue);
    const int64_t full = tiles / PLAN_PAIRS, rest = tiles % PLAN_PAIRS;
    double end = full * turn + (full ? at.delay : 0.0);
    const double last = (full + 1) * turn + (rest > at.early ? at.delay : 0.0);
    if (rest && last > end) end = last;
    const double cost = end + (products < epilogue ? products : epilogue) + LEAVE_CYCLES;
    if (p->cost == 0 || cost < p->cost) set_whole(tiles, cost, p);
}

// Tail tiles in parts: tiles_a of them in parts of per_a k-blocks for the early pairs, the
// others in parts of per_b for the late ones.
void plan_parts(int64_t tiles, int64_t tail, int64_t kb, double turn, Start at, int64_t tiles_a, int64_t per_a, int64_t per_b,
                Plan* p) {
    const int64_t sa = ceil_div(kb, per_a), sb = ceil_div(kb, per_b), tiles_b = tail - tiles_a, late = PLAN_PAIRS - at.early;
    const int64_t parts = tiles_a * sa + tiles_b * sb;
    const int64_t turns_a = ceil_div(tiles_a * sa, at.early), turns_b = tiles_b ? ceil_div(tiles_b * sb, late) : 0;
    double end = turns_a * (per_a * KB_CYCLES + FILL_CYCLES);
    const double end_b = at.delay + turns_b * (per_b * KB_CYCLES + FILL_CYCLES);
    if (late && end_b > end) end = end_b;
    const double cost = (tiles - tail) / PLAN_PAIRS * turn + end + LEAVE_CYCLES + FINISH_CYCLES + parts * PART_CYCLES;
    if (cost >= p->cost) return;
    memset(p, 0, sizeof(*p));
    p->cost = cost;
    p->split = {static_cast<int>(tiles - tail), PLAN_PAIRS,           at.early,
                static_cast<int>(tiles_a),      static_cast<int>(sa), static_cast<int>(per_a),
                static_cast<int>(sb),           static_cast<int>(per_b)};
    p->tail = static_cast<int>(tail);
    p->units = static_cast<int>(tiles - tail + (turns_a > turns_b ? turns_a : turns_b) * PLAN_PAIRS);
    p->part = static_cast<size_t>(parts) * 4 * PAIR_ROWS * PAIR_COLS;
}

// few: the kernels for few rows may run (A K-major, a 16-bit result); k_major: B is;
// epilogue: SM cycles that the epilogue of a whole tile of the pair kernel takes.
Plan plan_product(int64_t rows, int cols, int64_t k, bool few, bool k_major, double epilogue, Start at) {
    Plan p = {};
    const int64_t kb = ceil_div(k, GEMM_BK), tiles = tiles_of(rows, cols);
    // One or two tokens and a small weight: no tensor core, no join, half the latency.  Against
    // row_gemm_kernel, us: 2816 x 768 one token 2.7/4.4, two 3.4/4.5; 4096 x 4096 9.7/9.9 and 12.3/10;
    // 16384 x 4096 27/23.3.
    if (few && k_major && rows <= TOKEN_ROWS && rows * k <= TOKEN_CHUNKS * 8 && rows * rows * cols * k <= 1 << 24) {
        p.tokens = p.few = true;
        return p;
    }
    if (few && rows <= FEW_ROWS) plan_few(rows, cols, kb, epilogue, &p);
    plan_whole(tiles, kb, epilogue, at, &p);
    const double turn = turn_cycles(kb, epilogue);
    for (int64_t tail = tiles % PLAN_PAIRS;; tail = tiles) {
        if (tail && at.early == PLAN_PAIRS) {
            // parts beyond a few turns only add traffic
            for (int64_t s = 1; s <= 64 && s <= kb && tail * s <= 5 * PLAN_PAIRS; ++s)
                plan_parts(tiles, tail, kb, turn, at, tail, ceil_div(kb, s), kb, &p);
        } else if (tail) {
            // so many turns of the early pairs at so many parts, the rest in as many parts as fill
            // the late pairs for so many turns
            const int64_t late = PLAN_PAIRS - at.early;
            for (int64_t ta = 1; ta <= 4; ++ta)
                for (int64_t sa = 1; sa <= 16 && sa <= kb; ++sa) {
                    const int64_t most = ta * at.early / sa, tiles_a = most < tail ? most : tail, tiles_b = tail - tiles_a;
                    if (!tiles_a) break;
                    if (!tiles_b) {
                        plan_parts(tiles, tail, kb, turn, at, tiles_a, ceil_div(kb, sa), kb, &p);
                        continue;
                    }
                    for (int64_t tb = 1; tb <= 4; ++tb) {
                        int64_t sb = tb * late / tiles_b;
                        if (sb > 64) sb = 64;
                        if (sb > kb) sb = kb;
                        if (sb) plan_parts(tiles, tail, kb, turn, at, tiles_a, ceil_div(kb, sa), ceil_div(kb, sb), &p);
                    }
                }
        }
        if (tail == tiles) break;
    }
    return p;
}

// The two products of a backward pass.  The second kernel's pairs start where the first
// leaves SMs idle, so a last turn of the first that is not full costs nothing when the
// second's parts are cut to fill it; or both run as they would alone.
void plan_both(int64_t rows1, int cols1, int64_t k1, bool k_major1, double epilogue1, int64_t rows2, int cols2, int64_t k2,
               double epilogue2, Plan* first, Plan* second) {
    *first = plan_product(rows1, cols1, k1, true, k_major1, epilogue1, ALL_FREE);
    *second = plan_product(rows2, cols2, k2, false, false, epilogue2, ALL_FREE);
    if (first->few) return;
    const int64_t kb = ceil_div(k1, GEMM_BK), tiles = tiles_of(rows1, cols1);
    const int64_t full = tiles / PLAN_PAIRS, rest = tiles % PLAN_PAIRS;
    const double turn = turn_cycles(kb, epilogue1);
    const Start at = {rest ? static_cast<int>(PLAN_PAIRS - rest) : PLAN_PAIRS, rest ? turn : 0.0};
    const Plan p = plan_product(rows2, cols2, k2, false, false, epilogue2, at);
    const double cost = full * turn + LEAVE_CYCLES + p.cost;
    if (cost >= first->cost + second->cost) return;
    set_whole(tiles, full * turn + LEAVE_CYCLES, first);
    *second = p;
}

// The epilogue's cost for plan_product, by what it does: measured on 14336 x 6144 x 832
// (over the plain store) and, for arrays off the 16-byte boundaries, on 1000 x 2815 x 771.
double epilogue_cycles(const GemmEpilogue& e, int64_t rows) {
    const int es = e.out_f32 ? 4 : 2;
    double c = 2500.0;
    if (e.in) c += aligned16(e.in, e.ldin, es, rows) ? 2000.0 : 12000.0;
    if (e.z) c += aligned16(e.z, e.ldz, es, rows) ? 2500.0 : 12000.0;
    if (!aligned16(e.out, e.ldout, es, rows)) c += 12000.0;
    if (e.act == ACT_GELU || e.act == ACT_GELU_TANH) c += 6000.0;
    if (e.act == ACT_SILU) c += 3000.0;
    return c;
}

// Launches the product; what is left to add up of it goes to `rest`.
anvil_status run_product(const Product& q, const Plan& plan, DeviceState* dev, cudaStream_t s, TailSumParams* rest) {
    anvil_status st;
    cudaError_t e;
    if (plan.tokens) {
        TokenParams g;
        memset(&g, 0, sizeof(g));
        g.x = q.a.p;
        g.w = q.b.p;
        g.epi = q.epi;
        g.ldx = q.a.ld;
        g.ldw = q.b.ld;
        g.rows = static_cast<int>(q.rows);
        g.cols = q.cols;
        g.k = static_cast<int>(q.k);
        g.f16 = q.f16;
        e = profiled(ANVIL_KERNEL_LINEAR_PRODUCT, s, [&] { return launch_tokens(g, s); });
        return e ? cuda_fail(e, "linear product launch") : ANVIL_OK;
    }
    if (plan.few) {
        RowGemmParams g;
        memset(&g, 0, sizeof(g));
        // the output's columns run along B's rows: B is the M side of the MMA
        if ((st = encode(&g.tm_a, 2, q.f16, q.b.p, q.b.cols, q.b.rows, q.b.ld, 64, q.b_mn ? 64 : ROW_TILE_A))) return st;
        if ((st = encode(&g.tm_b, 2, q.f16, q.a.p, q.a.cols, q.a.rows, q.a.ld, 64, plan.bn))) return st;
        g.epi = q.epi;
        g.na = q.cols;
        g.nb = static_cast<int>(q.rows);
        g.k = static_cast<int>(q.k);
        g.a_mn = q.b_mn;
        g.f16 = q.f16;
        g.splits = plan.splits;
        g.kb_per_split = plan.kb;
        g.err = dev->err;
        e = profiled(ANVIL_KERNEL_LINEAR_PRODUCT, s, [&] { return launch_row_gemm(g, plan.bn, dev->sm_count, s); });
        return e ? cuda_fail(e, "linear product launch") : ANVIL_OK;
    }
    PairGemmParams g;
    memset(&g, 0, sizeof(g));
    if ((st = encode(&g.tm_a, 2, q.f16, q.a.p, q.a.cols, q.a.rows, q.a.ld, 64, q.a_mn ? 64 : 128))) return st;
    if ((st = encode(&g.tm_b, 2, q.f16, q.b.p, q.b.cols, q.b.rows, q.b.ld, 64, q.b_mn ? 64 : PAIR_COLS / 2))) return st;
    g.epi = q.epi;
    g.rows = static_cast<int>(q.rows);
    g.cols = q.cols;
    g.k = static_cast<int>(q.k);
    g.a_mn = q.a_mn;
    g.b_mn = q.b_mn;
    g.f16 = q.f16;
    g.tiles_r = static_cast<int>((q.rows + PAIR_ROWS - 1) / PAIR_ROWS);
    g.tiles_c = (q.cols + PAIR_COLS - 1) / PAIR_COLS;
    g.split = plan.split;
    g.units = plan.units;
    g.overlap_next = q.overlap_next;
    g.overlap_previous = q.overlap_previous;
    g.err = dev->err;
    const GemmEpilogue& ep = q.epi;
    const int es = ep.out_f32 ? 4 : 2;
    g.out_tma = aligned16(ep.out, ep.ldout, es, q.rows);
    g.in_tma = ep.in && aligned16(ep.in, ep.ldin, es, q.rows);
    g.z_tma = ep.z && aligned16(ep.z, ep.ldz, es, q.rows);
    // Half the staging makes room for a sixth stage: faster where the products bound it, slower
    // where the epilogue does.  Measured with six stages and five, us: 4096 x 50304 x 768 plain
    // 198/215, with residual 226/250, with stored z 298/267, off the 16-byte boundaries (50257 columns)
    // with residual 566/350; 14336 x 6144 x 832 plain 90/96; 30570 x 1872 x 104 plain 41/33.
    const bool products = q.k >= 8 * GEMM_BK && !ep.z && g.out_tma && (!ep.in || g.in_tma);
    g.box_bytes = products ? 64 : 128;
    const int box = g.box_bytes / es;  // columns of a staging box
    if (g.out_tma && (st = encode(&g.tm_out, es, q.f16, ep.out, q.cols, q.rows, ep.ldout, box, 128))) return st;
    if (g.in_tma && (st = encode(&g.tm_in, es, q.f16, ep.in, q.cols, q.rows, ep.ldin, box, 128))) return st;
    if (g.z_tma && (st = encode(&g.tm_z, es, q.f16, ep.z, q.cols, q.rows, ep.ldz, box, 128))) return st;
    if (plan.tail && (st = encode(&g.tm_part, 4, false, q.part, PAIR_COLS,
                                  static_cast<int64_t>(plan.part / (4 * PAIR_COLS)), PAIR_COLS, g.box_bytes / 4, 128)))
        return st;
    e = profiled(ANVIL_KERNEL_LINEAR_PRODUCT, s, [&] { return launch_pair_gemm(g, dev->sm_count, s); });
    if (e) return cuda_fail(e, "linear product launch");
    if (plan.tail) {
        rest->epi = ep;
        rest->part = q.part;
        rest->rows = g.rows;
        rest->cols = g.cols;
        rest->tiles_r = g.tiles_r;
        rest->tiles_c = g.tiles_c;
        rest->tiles = plan.tail;
        rest->split = plan.split;
    }
    return ANVIL_OK;
}

// The finishing launch, where there is anything to finish.
anvil_status run_finish(const FinishParams& f, cudaStream_t s) {
    if (!f.tail[0].tiles && !f.tail[1].tiles && !f.bias.out) return ANVIL_OK;
    const cudaError_t e = profiled(ANVIL_KERNEL_LINEAR_SUM, s, [&] { return launch_finish(f, s); });
    return e ? cuda_fail(e, "linear sum launch") : ANVIL_OK;
}

// Operands off the 16-byte boundaries become copies on them, in one launch.
struct Copies {
    RepackParams p;
    void add(Stored* s, void* copy) {
        if (!copy_bytes(*s)) return;
        const Stored to = with_copy(*s, copy);
        put(*s, copy, s->rows, to.ld);
        *s = to;
    }
    // s into `rows` rows at dst, ldd elements apart (rows and columns that s lacks: zeros)
    void put(const Stored& s, void* dst, int64_t rows, int64_t ldd) {
        Repack& r = p.job[p.jobs++];
        r.src = static_cast<const uint16_t*>(s.p);
        r.dst = static_cast<uint16_t*>(dst);
        r.rows = rows;
        r.src_rows = s.rows;
        r.lds = s.ld;
        r.cols = s.cols;
        r.ldd = ldd;
    }
    anvil_status run(cudaStream_t s) const {
        if (!p.jobs) return ANVIL_OK;
        const cudaError_t e = profiled(ANVIL_KERNEL_LINEAR_PREPARE, s, [&] { return launch_repack(p, s); });
        return e ? cuda_fail(e, "operand copy launch") : ANVIL_OK;
    }
};

Stored stored_weight(const void* w, int n, int k, int64_t ldw, bool transposed) {
    return transposed ? Stored{w, k, ldw, n} : Stored{w, n, ldw, k};
}

GemmEpilogue forward_epilogue(const anvil_linear_desc* d) {
    GemmEpilogue e = {};
    e.bias = d->bias;
    e.bias_f32 = d->bias && d->bias_dtype == ANVIL_F32;
    e.act = d->activation;
    e.in = d->residual;
    e.ldin = d->ldr;
    e.z = d->preact;
    e.ldz = d->ldz;
    e.out = d->y;
    e.ldout = d->ldy;
    return e;
}
GemmEpilogue dx_epilogue(const anvil_linear_grad_desc* d) {
    GemmEpilogue e = {};
    e.out = d->dx;
    e.ldout = d->lddx;
    return e;
}
GemmEpilogue dweight_epilogue(const anvil_linear_grad_desc* d) {
    GemmEpilogue e = {};
    e.out = d->dweight;
    e.ldout = d->lddw;
    e.out_f32 = d->dweight_dtype == ANVIL_F32;
    if (d->accumulate) {
        e.in = d->dweight;
        e.ldin = d->lddw;
    }
    return e;
}

struct LinearLayout {
    Stored x, w;
    Plan plan;
    size_t off_x, off_w, off_part, total;
};
LinearLayout linear_layout(const anvil_linear_desc* d) {
    LinearLayout L;
    L.x = {d->x, d->rows, d->ldx, d->k};
    L.w = stored_weight(d->weight, d->n, d->k, d->ldw, d->weight_transposed != 0);
    L.off_x = 0;
    L.off_w = L.off_x + copy_bytes(L.x);
    L.off_part = L.off_w + copy_bytes(L.w);
    const double cycles = epilogue_cycles(forward_epilogue(d), d->rows);
    L.plan = plan_product(d->rows, d->n, d->k, true, !d->weight_transposed, cycles, ALL_FREE);
    L.total = L.off_part + L.plan.part;
    return L;
}

anvil_status check_linear(const anvil_linear_desc* d) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    anvil_status st = check_linear_sizes(d->rows, d->n, d->k, d->dtype, d->activation);
    if (st != ANVIL_OK) return st;
    if (d->bias && d->bias_dtype != ANVIL_F32 && d->bias_dtype != d->dtype) return ANVIL_ERR_INVALID_ARG;
    if (d->rows == 0) return ANVIL_OK;
    if (!d->x || !d->weight || !d->y) return ANVIL_ERR_INVALID_ARG;
    const bool tr = d->weight_transposed != 0;
    if (bad_ld(d->rows, d->k, d->ldx) || bad_ld(tr ? d->k : d->n, tr ? d->n : d->k, d->ldw) || bad_ld(d->rows, d->n, d->ldy) ||
        (d->residual && bad_ld(d->rows, d->n, d->ldr)) || (d->preact && bad_ld(d->rows, d->n, d->ldz)))
        return ANVIL_ERR_INVALID_ARG;
    if (misaligned(d->x, 2) || misaligned(d->weight, 2) || misaligned(d->y, 2) || misaligned(d->residual, 2) ||
        misaligned(d->preact, 2) || (d->bias && misaligned(d->bias, size_of(d->bias_dtype))))
        return ANVIL_ERR_ALIGNMENT;
    return ANVIL_OK;
}

int grad_activation(const anvil_linear_grad_desc* d) { return d->activation & ~ANVIL_DZ_TWO_PARTS; }

// dz in two parts (h, the rounded values, and l, what that drops, rounded itself), for products that
// know one operand and one contraction: dz is stored as rows of h, then l, n8 = n rounded up to
// eights each.  For dx = (h + l) W a row is one row of 2 n8 columns, beside W twice; for
// dW = (h + l)^T x the same memory is 2 rows of n8 columns, beside every row of x twice.
struct LinearGradLayout {
    Stored dz, x, w;
    bool prep;        // act_grad_kernel runs
    bool dz_made;     // and writes dz
    bool two;         // in two parts
    int64_t n8;
    int64_t kdx, kdw; // contractions of the products
    Plan pdx, pdw;
    int rows_per_block, blocks_r;
    size_t off_dz, off_x, off_w, off_sum, off_part, total;
};

LinearGradLayout linear_grad_layout(const anvil_linear_grad_desc* d) {
    LinearGradLayout L;
    memset(&L, 0, sizeof(L));
    const bool tr = d->weight_transposed != 0;
    L.dz = {d->dy, d->rows, d->lddy, d->n};
    L.x = {d->x, d->rows, d->ldx, d->k};
    L.w = stored_weight(d->weight, d->n, d->k, d->ldw, tr);
    const bool products = d->dx || d->dweight;
    const bool act = grad_activation(d) != ANVIL_ACT_NONE;
    L.dz_made = products && (act || copy_bytes(L.dz) != 0);
    L.prep = L.dz_made || d->dbias;
    L.two = products && act && (d->activation & ANVIL_DZ_TWO_PARTS);
    L.n8 = (d->n + 7) & ~7;
    L.kdx = L.two ? 2 * L.n8 : d->n;
    L.kdw = L.two ? 2 * d->rows : d->rows;
    const int64_t k8 = (d->k + 7) & ~7;
    size_t at = 0;
    L.off_dz = at;
    if (L.dz_made) at += align256(2 * static_cast<size_t>(d->rows) * (L.two ? 2 : 1) * L.n8);
    L.off_x = at;
    if (d->dweight) at += L.two ? align256(2 * static_cast<size_t>(2 * d->rows) * k8) : copy_bytes(L.x);
    L.off_w = at;
    if (d->dx) at += L.two ? align256(2 * static_cast<size_t>(2 * L.n8) * (tr ? d->k : k8)) : copy_bytes(L.w);
    L.off_sum = at;
    if (L.prep) {
        // one turn of the blocks that the device holds at once, at least 32 rows each
        const int64_t cb = ceil_div(d->n, ACT_GRAD_COLS), most = ceil_div(d->rows, 32);
        int64_t br = ACT_GRAD_BLOCKS * PLAN_SMS / cb;
        if (br > most) br = most;
        if (br < 1) br = 1;
        L.rows_per_block = static_cast<int>((d->rows + br - 1) / br);
        L.blocks_r = static_cast<int>((d->rows + L.rows_per_block - 1) / L.rows_per_block);
        if (d->dbias) at += align256(sizeof(float) * static_cast<size_t>(L.blocks_r) * d->n);
    }
    L.off_part = at;
    const int64_t wr = tr ? d->k : d->n;
    const int wc = tr ? d->n : d->k;
    const double ex = epilogue_cycles(dx_epilogue(d), d->rows), ew = epilogue_cycles(dweight_epilogue(d), wr);
    if (d->dx && d->dweight) plan_both(d->rows, d->k, L.kdx, tr, ex, wr, wc, L.kdw, ew, &L.pdx, &L.pdw);
    else if (d->dx) L.pdx = plan_product(d->rows, d->k, L.kdx, true, tr, ex, ALL_FREE);
    else if (d->dweight) L.pdw = plan_product(wr, wc, L.kdw, false, false, ew, ALL_FREE);
    L.total = at + L.pdx.part + L.pdw.part;  // the second product may start before the first's parts are added up
    return L;
}

anvil_status check_linear_grad(const anvil_linear_grad_desc* d) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    anvil_status st = check_linear_sizes(d->rows, d->n, d->k, d->dtype, grad_activation(d));
    if (st != ANVIL_OK) return st;
    if ((d->activation & ANVIL_DZ_TWO_PARTS) && d->rows > ANVIL_MAX_ROWS / 2) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    if (d->dweight && d->dweight_dtype != ANVIL_F32 && d->dweight_dtype != d->dtype) return ANVIL_ERR_INVALID_ARG;
    const bool tr = d->weight_transposed != 0;
    if (d->dweight && bad_ld(tr ? d->k : d->n, tr ? d->n : d->k, d->lddw)) return ANVIL_ERR_INVALID_ARG;
    if ((d->dweight && misaligned(d->dweight, size_of(d->dweight_dtype))) || misaligned(d->dbias, 4))
        return ANVIL_ERR_ALIGNMENT;
    if (d->rows == 0) return ANVIL_OK;
    if (!d->dx && !d->dweight && !d->dbias) return ANVIL_OK;
    const bool act = grad_activation(d) != ANVIL_ACT_NONE;
    if (!d->dy || (d->dweight && !d->x) || (d->dx && !d->weight) || (act && !d->preact)) return ANVIL_ERR_INVALID_ARG;
    if (bad_ld(d->rows, d->n, d->lddy) || (d->dweight && bad_ld(d->rows, d->k, d->ldx)) ||
        (d->dx && (bad_ld(tr ? d->k : d->n, tr ? d->n : d->k, d->ldw) || bad_ld(d->rows, d->k, d->lddx))) ||
        (act && bad_ld(d->rows, d->n, d->ldz)))
        return ANVIL_ERR_INVALID_ARG;
    if (misaligned(d->dy, 2) || misaligned(d->x, 2) || misaligned(d->weight, 2) || misaligned(d->preact, 2) ||
        misaligned(d->dx, 2))
        return ANVIL_ERR_ALIGNMENT;
    return ANVIL_OK;
}

}  // namespace

extern "C" {

anvil_status anvil_layernorm_forward(const anvil_layernorm_desc* d, void* stream) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    anvil_status st = check_norm_sizes(d->rows, d->width, d->dtype, d->weight_dtype);
    if (st != ANVIL_OK) return st;
    if (d->rows == 0) return ANVIL_OK;
    if (!d->x || !d->y || bad_ld(d->rows, d->width, d->ldx) || bad_ld(d->rows, d->width, d->ldy)) return ANVIL_ERR_INVALID_ARG;
    const int es = size_of(d->dtype), ws = size_of(d->weight_dtype);
    if (misaligned(d->x, es) || misaligned(d->y, es) || misaligned(d->weight, ws) || misaligned(d->bias, ws) ||
        misaligned(d->mean, 4) || misaligned(d->rstd, 4))
        return ANVIL_ERR_ALIGNMENT;
    const Area a[6] = {area(d->x, d->rows, d->width, d->ldx, es, false), area(d->weight, 1, d->width, 0, ws, false),
                       area(d->bias, 1, d->width, 0, ws, false),         area(d->y, d->rows, d->width, d->ldy, es, true),
                       area(d->mean, 1, d->rows, 0, 4, true),            area(d->rstd, 1, d->rows, 0, 4, true)};
    const int inplace[1][2] = {{3, 0}};
    if ((st = check_areas(a, 6, inplace, 1)) != ANVIL_OK) return st;
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    NormFwdParams p;
    p.x = d->x;
    p.weight = d->weight;
    p.bias = d->bias;
    p.y = d->y;
    p.mean = d->mean;
    p.rstd = d->rstd;
    p.rows = d->rows;
    p.ldx = d->ldx;
    p.ldy = d->ldy;
    p.width = d->width;
    p.dtype = d->dtype;
    p.weight_dtype = d->weight_dtype;
    p.eps = d->eps;
    p.team_rows = 0;
    p.err = dev->err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = profiled(ANVIL_KERNEL_NORM_FORWARD, s, [&] { return launch_norm_fwd(p, s); });
    return e ? cuda_fail(e, "layer norm launch") : ANVIL_OK;
}

size_t anvil_layernorm_backward_workspace_bytes(const anvil_layernorm_grad_desc* d) {
    if (!d || check_norm_sizes(d->rows, d->width, d->dtype, d->weight_dtype) != ANVIL_OK) return 0;
    return norm_bwd_bytes(d);
}

anvil_status anvil_layernorm_backward(const anvil_layernorm_grad_desc* d, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    anvil_status st = check_norm_sizes(d->rows, d->width, d->dtype, d->weight_dtype);
    if (st != ANVIL_OK) return st;
    if (!d->dx && !d->dweight && !d->dbias) return ANVIL_OK;
    if (misaligned(d->dweight, 4) || misaligned(d->dbias, 4)) return ANVIL_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    DeviceState* dev = nullptr;
    if (d->rows == 0) {
        if (!d->dweight && !d->dbias) return ANVIL_OK;
        if ((st = device_setup(&dev)) != ANVIL_OK) return st;
        if ((d->dweight && (e = cudaMemsetAsync(d->dweight, 0, sizeof(float) * d->width, s))) ||
            (d->dbias && (e = cudaMemsetAsync(d->dbias, 0, sizeof(float) * d->width, s))))
            return cuda_fail(e, "cudaMemsetAsync");
        return ANVIL_OK;
    }
    if (!d->dy || !d->x || !d->mean || !d->rstd || bad_ld(d->rows, d->width, d->lddy) || bad_ld(d->rows, d->width, d->ldx) ||
        (d->dx && bad_ld(d->rows, d->width, d->lddx)) || (d->residual_grad && bad_ld(d->rows, d->width, d->ldr)))
        return ANVIL_ERR_INVALID_ARG;
    const int es = size_of(d->dtype), ws = size_of(d->weight_dtype);
    if (misaligned(d->dy, es) || misaligned(d->x, es) || misaligned(d->dx, es) || misaligned(d->residual_grad, es) ||
        misaligned(d->weight, ws) || misaligned(d->mean, 4) || misaligned(d->rstd, 4))
        return ANVIL_ERR_ALIGNMENT;
    const Area a[9] = {area(d->dy, d->rows, d->width, d->lddy, es, false),
                       area(d->x, d->rows, d->width, d->ldx, es, false),
                       area(d->mean, 1, d->rows, 0, 4, false),
                       area(d->rstd, 1, d->rows, 0, 4, false),
                       area(d->weight, 1, d->width, 0, ws, false),
                       area(d->residual_grad, d->rows, d->width, d->ldr, es, false),
                       area(d->dx, d->rows, d->width, d->lddx, es, true),
                       area(d->dweight, 1, d->width, 0, 4, true),
                       area(d->dbias, 1, d->width, 0, 4, true)};
    const int inplace[3][2] = {{6, 0}, {6, 1}, {6, 5}};
    if ((st = check_areas(a, 9, inplace, 3)) != ANVIL_OK) return st;
    const size_t need = norm_bwd_bytes(d);
    if ((st = check_workspace(workspace, workspace_bytes, need, a, 9)) != ANVIL_OK) return st;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    NormBwdParams p;
    p.dy = d->dy;
    p.x = d->x;
    p.mean = d->mean;
    p.rstd = d->rstd;
    p.weight = d->weight;
    p.res = d->dx ? d->residual_grad : nullptr;
    p.dx = d->dx;
    p.dweight = d->dweight;
    p.dbias = d->dbias;
    p.part = static_cast<float*>(workspace);
    p.rows = d->rows;
    p.lddy = d->lddy;
    p.ldx = d->ldx;
    p.ldr = d->ldr;
    p.lddx = d->lddx;
    p.width = d->width;
    p.dtype = d->dtype;
    p.weight_dtype = d->weight_dtype;
    p.err = dev->err;
    norm_bwd_plan(&p);
    if ((e = profiled(ANVIL_KERNEL_NORM_BACKWARD, s, [&] { return launch_norm_bwd(p, s); })))
        return cuda_fail(e, "layer norm gradient launch");
    if (p.blocks > 1 && (p.dweight || p.dbias) &&
        (e = profiled(ANVIL_KERNEL_NORM_GRADS, s, [&] { return launch_norm_grads(p, s); })))
        return cuda_fail(e, "layer norm gradient launch");
    return ANVIL_OK;
}

size_t anvil_linear_workspace_bytes(const anvil_linear_desc* d) {
    if (check_linear(d) != ANVIL_OK || d->rows == 0) return 0;
    return linear_layout(d).total;
}

anvil_status anvil_linear_forward(const anvil_linear_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
    anvil_status st = check_linear(d);
    if (st != ANVIL_OK || d->rows == 0) return st;
    const bool tr = d->weight_transposed != 0;
    const int bs = d->bias ? size_of(d->bias_dtype) : 2;
    const Area a[6] = {area(d->x, d->rows, d->k, d->ldx, 2, false),
                       area(d->weight, tr ? d->k : d->n, tr ? d->n : d->k, d->ldw, 2, false),
                       area(d->bias, 1, d->n, 0, bs, false),
                       area(d->residual, d->rows, d->n, d->ldr, 2, false),
                       area(d->y, d->rows, d->n, d->ldy, 2, true),
                       area(d->preact, d->rows, d->n, d->ldz, 2, true)};
    const int inplace[1][2] = {{4, 3}};
    if ((st = check_areas(a, 6, inplace, 1)) != ANVIL_OK) return st;
    LinearLayout L = linear_layout(d);
    if ((st = check_workspace(workspace, workspace_bytes, L.total, a, 6)) != ANVIL_OK) return st;
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Copies copies = {};
    copies.add(&L.x, ws + L.off_x);
    copies.add(&L.w, ws + L.off_w);
    if ((st = copies.run(s)) != ANVIL_OK) return st;
    Product q;
    memset(&q, 0, sizeof(q));
    q.a = L.x;
    q.b = L.w;
    q.b_mn = tr;
    q.rows = d->rows;
    q.cols = d->n;
    q.k = d->k;
    q.f16 = d->dtype == ANVIL_F16;
    q.epi = forward_epilogue(d);
    q.part = reinterpret_cast<float*>(ws + L.off_part);
    FinishParams f;
    memset(&f, 0, sizeof(f));
    f.f16 = q.f16;
    if ((st = run_product(q, L.plan, dev, s, &f.tail[0])) != ANVIL_OK) return st;
    return run_finish(f, s);
}

size_t anvil_linear_backward_workspace_bytes(const anvil_linear_grad_desc* d) {
    if (check_linear_grad(d) != ANVIL_OK || d->rows == 0) return 0;
    return linear_grad_layout(d).total;
}

anvil_status anvil_linear_backward(const anvil_linear_grad_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
    anvil_status st = check_linear_grad(d);
    if (st != ANVIL_OK) return st;
    if (!d->dx && !d->dweight && !d->dbias) return ANVIL_OK;
    const bool tr = d->weight_transposed != 0;
    const int dws = size_of(d->dweight_dtype);
    const int64_t wr = tr ? d->k : d->n, wc = tr ? d->n : d->k;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    DeviceState* dev = nullptr;
    if (d->rows == 0) {
        if (d->accumulate || (!d->dweight && !d->dbias)) return ANVIL_OK;
        if ((st = device_setup(&dev)) != ANVIL_OK) return st;
        if ((d->dweight && (e = cudaMemset2DAsync(d->dweight, (wr > 1 ? d->lddw : wc) * dws, 0, wc * dws, wr, s))) ||
            (d->dbias && (e = cudaMemsetAsync(d->dbias, 0, sizeof(float) * d->n, s))))
            return cuda_fail(e, "cudaMemsetAsync");
        return ANVIL_OK;
    }
    const bool act = grad_activation(d) != ANVIL_ACT_NONE;
    const Area a[7] = {area(d->dy, d->rows, d->n, d->lddy, 2, false),
                       area(d->dweight ? d->x : nullptr, d->rows, d->k, d->ldx, 2, false),
                       area(d->dx ? d->weight : nullptr, wr, wc, d->ldw, 2, false),
                       area(act ? d->preact : nullptr, d->rows, d->n, d->ldz, 2, false),
                       area(d->dx, d->rows, d->k, d->lddx, 2, true),
                       area(d->dweight, wr, wc, d->lddw, dws, true),
                       area(d->dbias, 1, d->n, 0, 4, true)};
    if ((st = check_areas(a, 7, nullptr, 0)) != ANVIL_OK) return st;
    LinearGradLayout L = linear_grad_layout(d);
    if ((st = check_workspace(workspace, workspace_bytes, L.total, a, 7)) != ANVIL_OK) return st;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool f16 = d->dtype == ANVIL_F16;
    FinishParams f;
    memset(&f, 0, sizeof(f));
    f.f16 = f16;
    if (L.prep) {
        ActGradParams p;
        memset(&p, 0, sizeof(p));
        p.dy = d->dy;
        p.z = act ? d->preact : nullptr;
        p.dz = L.dz_made ? ws + L.off_dz : nullptr;
        p.part = d->dbias ? reinterpret_cast<float*>(ws + L.off_sum) : nullptr;
        p.rows = d->rows;
        p.lddy = d->lddy;
        p.ldz = d->ldz;
        p.cols = d->n;
        p.act = grad_activation(d);
        p.two_parts = L.two;
        p.f16 = f16;
        p.rows_per_block = L.rows_per_block;
        p.blocks_r = L.blocks_r;
        if (L.dz_made) {
            L.dz = with_copy(L.dz, ws + L.off_dz);
            p.ldd = L.two ? 2 * L.n8 : L.dz.ld;
        }
        if ((e = profiled(ANVIL_KERNEL_LINEAR_PREPARE, s, [&] { return launch_act_grad(p, s); })))
            return cuda_fail(e, "activation gradient launch");
        f.bias = {p.part, d->dbias, p.blocks_r, d->n, d->accumulate};
    }
    Copies copies = {};
    Stored dz_dx = L.dz, dz_dw = L.dz;
    if (L.two) {
        dz_dx = {L.dz.p, d->rows, 2 * L.n8, static_cast<int>(2 * L.n8)};
        dz_dw.rows = 2 * d->rows;
        if (d->dx) {
            uint16_t* w2 = reinterpret_cast<uint16_t*>(ws + L.off_w);
            const Stored to = tr ? Stored{w2, d->k, 2 * L.n8, static_cast<int>(2 * L.n8)} : Stored{w2, 2 * L.n8, (d->k + 7) & ~7, d->k};
            copies.put(L.w, w2, tr ? d->k : L.n8, to.ld);
            copies.put(L.w, w2 + (tr ? L.n8 : L.n8 * to.ld), tr ? d->k : L.n8, to.ld);
            L.w = to;
        }
        if (d->dweight) {
            uint16_t* x2 = reinterpret_cast<uint16_t*>(ws + L.off_x);
            const Stored to = {x2, 2 * d->rows, (d->k + 7) & ~7, d->k};
            copies.put(L.x, x2, d->rows, 2 * to.ld);
            copies.put(L.x, x2 + to.ld, d->rows, 2 * to.ld);
            L.x = to;
        }
    } else {
        if (d->dx) copies.add(&L.w, ws + L.off_w);
        if (d->dweight) copies.add(&L.x, ws + L.off_x);
    }
    if ((st = copies.run(s)) != ANVIL_OK) return st;
    const bool overlap = d->dx && d->dweight && !L.pdx.few;
    if (d->dx) {
        Product q;
        memset(&q, 0, sizeof(q));
        q.a = dz_dx;
        q.b = L.w;
        q.b_mn = !tr;
        q.rows = d->rows;
        q.cols = d->k;
        q.k = L.kdx;
        q.f16 = f16;
        q.epi = dx_epilogue(d);
        q.part = reinterpret_cast<float*>(ws + L.off_part);
        q.overlap_next = overlap;
        if ((st = run_product(q, L.pdx, dev, s, &f.tail[0])) != ANVIL_OK) return st;
    }
    if (d->dweight) {
        Product q;
        memset(&q, 0, sizeof(q));
        q.a = tr ? L.x : dz_dw;
        q.b = tr ? dz_dw : L.x;
        q.a_mn = q.b_mn = true;
        q.rows = wr;
        q.cols = static_cast<int>(wc);
        q.k = L.kdw;
        q.f16 = f16;
        q.epi = dweight_epilogue(d);
        q.part = reinterpret_cast<float*>(ws + L.off_part + L.pdx.part);
        q.overlap_previous = overlap;
        if ((st = run_product(q, L.pdw, dev, s, &f.tail[1])) != ANVIL_OK) return st;
    }
    return run_finish(f, s);
}

anvil_status anvil_token_logprobs(const anvil_logprob_desc* d, void* stream) {
    if (!d || d->rows < 0 || d->vocab < 1 || !valid_dtype(d->dtype) || d->top < 0 || d->top > ANVIL_MAX_TOP ||
        d->top > d->vocab)
        return ANVIL_ERR_INVALID_ARG;
    if (d->rows > ANVIL_MAX_ROWS || d->vocab > ANVIL_MAX_VOCAB) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    if (d->rows == 0) return ANVIL_OK;
    if (!d->logits || bad_ld(d->rows, d->vocab, d->ld) || (d->logprob && !d->targets) ||
        (d->top && (!d->top_logprob || !d->top_index)))
        return ANVIL_ERR_INVALID_ARG;
    const int es = size_of(d->dtype), ts = d->targets_int64 ? 8 : 4;
    if (misaligned(d->logits, es) || misaligned(d->targets, ts) || misaligned(d->logprob, 4) || misaligned(d->entropy, 4) ||
        misaligned(d->lse, 4) || misaligned(d->top_logprob, 4) || misaligned(d->top_index, 4))
        return ANVIL_ERR_ALIGNMENT;
    const int64_t nt = d->rows * d->top;
    const Area a[7] = {area(d->logits, d->rows, d->vocab, d->ld, es, false),
                       area(d->targets, 1, d->rows, 0, ts, false),
                       area(d->logprob, 1, d->rows, 0, 4, true),
                       area(d->entropy, 1, d->rows, 0, 4, true),
                       area(d->lse, 1, d->rows, 0, 4, true),
                       area(d->top ? d->top_logprob : nullptr, 1, nt, 0, 4, true),
                       area(d->top ? d->top_index : nullptr, 1, nt, 0, 4, true)};
    anvil_status st;
    if ((st = check_areas(a, 7, nullptr, 0)) != ANVIL_OK) return st;
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    LogprobParams p;
    p.logits = d->logits;
    p.targets = d->targets;
    p.logprob = d->logprob;
    p.entropy = d->entropy;
    p.lse = d->lse;
    p.top_logprob = d->top_logprob;
    p.top_index = d->top_index;
    p.rows = d->rows;
    p.ld = d->ld;
    p.vocab = d->vocab;
    p.top = d->top;
    p.dtype = d->dtype;
    p.target64 = d->targets_int64 != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = profiled(ANVIL_KERNEL_LOGPROB, s, [&] { return launch_logprob_fwd(p, dev->sm_count, s); });
    return e ? cuda_fail(e, "token log-probability launch") : ANVIL_OK;
}

anvil_status anvil_token_logprobs_backward(const anvil_logprob_grad_desc* d, void* stream) {
    if (!d || d->rows < 0 || d->vocab < 1 || !valid_dtype(d->dtype)) return ANVIL_ERR_INVALID_ARG;
    if (d->rows > ANVIL_MAX_ROWS || d->vocab > ANVIL_MAX_VOCAB || d->rows * logprob_bwd_segments(d->vocab, d->dtype) > INT32_MAX)
        return ANVIL_ERR_UNSUPPORTED_SHAPE;
    if (d->rows == 0) return ANVIL_OK;
    if (!d->logits || !d->dlogits || !d->lse || (d->grad_logprob && !d->targets) || (d->grad_entropy && !d->entropy) ||
        bad_ld(d->rows, d->vocab, d->ld) || bad_ld(d->rows, d->vocab, d->ldd))
        return ANVIL_ERR_INVALID_ARG;
    const int es = size_of(d->dtype), ts = d->targets_int64 ? 8 : 4;
    if (misaligned(d->logits, es) || misaligned(d->dlogits, es) || misaligned(d->targets, ts) || misaligned(d->lse, 4) ||
        misaligned(d->entropy, 4) || misaligned(d->grad_logprob, 4) || misaligned(d->grad_entropy, 4))
        return ANVIL_ERR_ALIGNMENT;
    const Area a[7] = {area(d->logits, d->rows, d->vocab, d->ld, es, false),
                       area(d->targets, 1, d->rows, 0, ts, false),
                       area(d->lse, 1, d->rows, 0, 4, false),
                       area(d->entropy, 1, d->rows, 0, 4, false),
                       area(d->grad_logprob, 1, d->rows, 0, 4, false),
                       area(d->grad_entropy, 1, d->rows, 0, 4, false),
                       area(d->dlogits, d->rows, d->vocab, d->ldd, es, true)};
    const int inplace[1][2] = {{6, 0}};
    anvil_status st;
    if ((st = check_areas(a, 7, inplace, 1)) != ANVIL_OK) return st;
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    LogprobGradParams p;
    p.logits = d->logits;
    p.targets = d->targets;
    p.lse = d->lse;
    p.entropy = d->entropy;
    p.grad_logprob = d->grad_logprob;
    p.grad_entropy = d->grad_entropy;
    p.dlogits = d->dlogits;
    p.rows = d->rows;
    p.ld = d->ld;
    p.ldd = d->ldd;
    p.vocab = d->vocab;
    p.dtype = d->dtype;
    p.target64 = d->targets_int64 != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = profiled(ANVIL_KERNEL_LOGPROB_BACKWARD, s, [&] { return launch_logprob_bwd(p, s); });
    return e ? cuda_fail(e, "token log-probability gradient launch") : ANVIL_OK;
}

}  // extern "C"
