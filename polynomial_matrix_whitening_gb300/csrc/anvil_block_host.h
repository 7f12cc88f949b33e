// anvil_block_host.h -- what the C ABI of the operators around the banks shares on the host: argument
// checks, tensor maps, the plan of a product (which kernel, which tile shape, how split) and its launch
// (internal to libanvil).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/anvil.h"
#include "anvil_host.h"
#include "anvil_linear.h"

namespace anvil {

inline int size_of(int dtype) { return dtype == ANVIL_F32 ? 4 : 2; }
inline bool valid_dtype(int dtype) { return dtype == ANVIL_F32 || dtype == ANVIL_BF16 || dtype == ANVIL_F16; }

// A row-major array of the call: `rows` rows of `width` bytes, `ld` bytes apart.
struct Area {
    uintptr_t p;
    int64_t rows, ld, width;
    bool written;
};

inline Area area(const void* p, int64_t rows, int64_t cols, int64_t ld, int es, bool written) {
    return {reinterpret_cast<uintptr_t>(p), rows, rows > 1 ? ld * es : cols * es, cols * es, written};
}

// Whether two areas share a byte.  Interleaved rows (the same row stride) share none when
// their columns are disjoint; other areas are taken as the whole range they span.
inline bool share(const Area& a, const Area& b) {
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
inline bool same(const Area& a, const Area& b) { return a.p == b.p && a.rows == b.rows && a.ld == b.ld && a.width == b.width; }

// Every written area against every other; `inplace` lists the pairs (written, other) that
// may be the very same array.
inline anvil_status check_areas(const Area* a, int n, const int (*inplace)[2], int npairs) {
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

inline bool misaligned(const void* p, int es) { return (reinterpret_cast<uintptr_t>(p) & (es - 1)) != 0; }
inline bool bad_ld(int64_t rows, int64_t cols, int64_t ld) { return rows > 1 && ld < cols; }

inline anvil_status check_workspace(const void* ws, size_t bytes, size_t need, const Area* a, int n) {
    if (need == 0) return ANVIL_OK;
    if (!ws || bytes < need) return ANVIL_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255) return ANVIL_ERR_ALIGNMENT;
    const Area w = {reinterpret_cast<uintptr_t>(ws), 1, static_cast<int64_t>(need), static_cast<int64_t>(need), true};
    for (int i = 0; i < n; ++i)
        if (share(w, a[i])) return ANVIL_ERR_ALIAS;
    return ANVIL_OK;
}

// The SM count the work is divided for (a GB300's; one constant, so that the workspaces need
// no device query and the order of the sums is the same everywhere).
constexpr int PLAN_SMS = 152;

// ---------------------------------------------------------------- products
inline anvil_status check_linear_sizes(int64_t rows, int n, int k, int dtype, int act) {
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
inline size_t copy_bytes(const Stored& s) {
    if (aligned16(s.p, s.ld, 2, s.rows)) return 0;
    return align256(2 * static_cast<size_t>(s.rows) * ((s.cols + 7) & ~7));
}
inline Stored with_copy(const Stored& s, void* copy) {
    Stored r = s;
    r.p = copy;
    r.ld = (s.cols + 7) & ~7;
    return r;
}

// Tensor map of a row-major matrix [outer][inner], boxes of box1 rows by box0 elements
// (128 or 64 bytes, the swizzle of that size).  A third dimension of one, for the 3-D copies.
inline anvil_status encode(CUtensorMap* map, int es, bool f16, const void* base, int64_t inner, int64_t outer, int64_t ld, int box0,
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
    bool one_chain, overlap_next, overlap_previous;  // pair_gemm_kernel's flags
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

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Blocks of 128 weight rows by 16 to 128 tokens, the contraction whole or split over a
// cluster.  Estimated times in SM cycles, from the kernel's own time stamps: 545 for a
// k-block (the MMA reads its 128-row operand at 32 bytes a cycle, whatever the tokens),
// 1700 to the first and from the last, 28 for a token's column; a join 2500, and 250 for
// a token's column of each block's share.
inline void plan_few(int64_t rows, int cols, int64_t kb, double epilogue, Plan* p) {
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

inline int64_t tiles_of(int64_t rows, int cols) { return ceil_div(rows, PAIR_ROWS) * ceil_div(cols, PAIR_COLS); }
inline double turn_cycles(int64_t kb, double epilogue) { return kb * KB_CYCLES > epilogue ? kb * KB_CYCLES : epilogue; }

inline void set_whole(int64_t tiles, double cost, Plan* p) {
    memset(p, 0, sizeof(*p));
    p->cost = cost;
    p->split = {static_cast<int>(tiles), PLAN_PAIRS, PLAN_PAIRS, 0, 1, 0, 1, 0};
    p->units = static_cast<int>(tiles);
}

inline void plan_whole(int64_t tiles, int64_t kb, double epilogue, Start at, Plan* p) {
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
inline void plan_parts(int64_t tiles, int64_t tail, int64_t kb, double turn, Start at, int64_t tiles_a, int64_t per_a, int64_t per_b,
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

// One or two tokens and a small weight: no tensor core, no join, half the latency.  Against
// row_gemm_kernel, us: 2816 x 768 one token 2.7/4.4, two 3.4/4.5; 4096 x 4096 9.7/9.9 and 12.3/10;
// 16384 x 4096 27/23.3.
inline bool token_product(int64_t rows, int cols, int64_t k) {
    return rows <= TOKEN_ROWS && rows * k <= TOKEN_CHUNKS * 8 && rows * rows * cols * k <= 1 << 24;
}

// The row kernel for `rows` tokens, up to 32 a tile, and so many tiles of the weight: split along k as long as
// two of its blocks share an SM at most and every part has four k-blocks (us in one part/two/four: gated 32 x 8192
// x 1024, 128 tiles, 9.7/8.5/14.6; 32 x 11008 x 4096, 172 tiles, 34.8/42; 16 x 5000 x 128, 79 tiles, 3.9/5.2; the
// head's 16 x 8000 x 4096, 63 tiles, 25.7/19.1/17.9).  Clusters of eight find fewer places: 64 blocks at most.
constexpr int ROW_TOKENS = 32;
inline int64_t row_tiles(int64_t rows) { return ceil_div(rows, rows <= 16 ? 16 : ROW_TOKENS); }
inline void set_rows(int64_t rows, int64_t weight_tiles, int64_t kb, Plan* p) {
    const int64_t blocks = weight_tiles * row_tiles(rows);
    memset(p, 0, sizeof(*p));
    p->few = true;
    p->bn = rows <= 16 ? 16 : ROW_TOKENS;
    p->splits = 1;
    for (int s = 2; s <= 8; s *= 2) {
        const int64_t per = ceil_div(kb, s);
        if (blocks * s > (s < 8 ? 2 * PLAN_SMS : 64) || per < 4 || per * (s - 1) >= kb) break;  // (every part has work)
        p->splits = s;
    }
    p->kb = static_cast<int>(ceil_div(kb, p->splits));
}

// few: the kernels for few rows may run (A K-major, a 16-bit result); k_major: B is;
// epilogue: SM cycles that the epilogue of a whole tile of the pair kernel takes.
inline Plan plan_product(int64_t rows, int cols, int64_t k, bool few, bool k_major, double epilogue, Start at) {
    Plan p = {};
    const int64_t kb = ceil_div(k, GEMM_BK), tiles = tiles_of(rows, cols);
    if (few && k_major && token_product(rows, cols, k)) {
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
// few1: the kernels for few rows may run the first.
inline void plan_both(int64_t rows1, int cols1, int64_t k1, bool few1, bool k_major1, double epilogue1, int64_t rows2, int cols2,
                      int64_t k2, double epilogue2, Plan* first, Plan* second) {
    *first = plan_product(rows1, cols1, k1, few1, k_major1, epilogue1, ALL_FREE);
    *second = plan_product(rows2, cols2, k2, false, false, epilogue2, ALL_FREE);
    if (first->few) return;
    const int64_t kb = ceil_div(k1, GEMM_BK), tiles = tiles_of(rows1, cols1);
    const int64_t full = tiles / PLAN_PAIRS, rest = tiles % PLAN_PAIRS;
    const double turn = turn_cycles(kb, epilogue1);
    const Start at = {rest ? static_cast<int>(PLAN_PAIRS - rest) : PLAN_PAIRS, rest ? turn : 0.0};
    const Plan p = plan_product(rows2, cols2, k2, false, false, epilogue2, at);
    double cost = full * turn + LEAVE_CYCLES + p.cost;
    // a last turn that is long beside the second product (a few tiles of a long contraction)
    const double alone = (full + (rest ? 1 : 0)) * turn + LEAVE_CYCLES;
    if (!few1 && alone > cost) cost = alone;
    if (cost >= first->cost + second->cost) return;
    set_whole(tiles, full * turn + LEAVE_CYCLES, first);
    *second = p;
}

// The epilogue's cost for plan_product, by what it does: measured on 14336 x 6144 x 832
// (over the plain store) and, for arrays off the 16-byte boundaries, on 1000 x 2815 x 771.
inline double epilogue_cycles(const GemmEpilogue& e, int64_t rows) {
    const int es = e.out_f32 ? 4 : 2;
    double c = 2500.0;
    if (e.in) c += aligned16(e.in, e.ldin, es, rows) ? 2000.0 : 12000.0;
    if (e.z) c += aligned16(e.z, e.ldz, es, rows) ? 2500.0 : 12000.0;
    if (!aligned16(e.out, e.ldout, es, rows)) c += 12000.0;
    if (e.act == ACT_GELU || e.act == ACT_GELU_TANH) c += 6000.0;
    if (e.act == ACT_SILU) c += 3000.0;
    return c;
}

// The pair kernel's parameters for one product; e2: a second result, which goes the same way.
inline anvil_status fill_pair(const Product& q, const Plan& plan, DeviceState* dev, PairGemmParams* to,
                              const GemmEpilogue* e2 = nullptr) {
    PairGemmParams& g = *to;
    anvil_status st;
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
    g.one_chain = q.one_chain;
    g.overlap_next = q.overlap_next;
    g.overlap_previous = q.overlap_previous;
    g.err = dev->err;
    const GemmEpilogue& ep = q.epi;
    const int es = ep.out_f32 ? 4 : 2;
    g.out_tma = aligned16(ep.out, ep.ldout, es, q.rows) && (!e2 || aligned16(e2->out, e2->ldout, es, q.rows));
    g.in_tma = ep.in && aligned16(ep.in, ep.ldin, es, q.rows) && (!e2 || aligned16(e2->in, e2->ldin, es, q.rows));
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
    return ANVIL_OK;
}
inline void fill_rest(const Product& q, const Plan& plan, const PairGemmParams& g, TailSumParams* rest) {
    rest->epi = q.epi;
    rest->part = q.part;
    rest->rows = g.rows;
    rest->cols = g.cols;
    rest->tiles_r = g.tiles_r;
    rest->tiles_c = g.tiles_c;
    rest->tiles = plan.tail;
    rest->split = plan.split;
}

// Launches the product; what is left to add up of it goes to `rest`.
inline anvil_status run_product(const Product& q, const Plan& plan, DeviceState* dev, cudaStream_t s, TailSumParams* rest) {
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
    if ((st = fill_pair(q, plan, dev, &g)) != ANVIL_OK) return st;
    e = profiled(ANVIL_KERNEL_LINEAR_PRODUCT, s, [&] { return launch_pair_gemm(g, dev->sm_count, s); });
    if (e) return cuda_fail(e, "linear product launch");
    if (plan.tail) fill_rest(q, plan, g, rest);
    return ANVIL_OK;
}

// Several products in one launch (PairMultiParams).  The operands of number result * segments +
// segment are a[i] and b[i], in q's order and of q's sizes; q.k is a segment's contraction, q.rows a
// result's rows.
struct MultiProduct {
    Product q;  // its a and b are number 0
    Stored a[4], b[4];
    int results, segments;
    GemmEpilogue epi2;
};
inline int64_t multi_k(int64_t k, int segments) { return segments * ceil_div(k, GEMM_BK) * GEMM_BK; }
// Rows that give plan_product the tiles of both results.
inline int64_t multi_rows(int64_t rows, int results) { return results > 1 ? results * ceil_div(rows, PAIR_ROWS) * PAIR_ROWS : rows; }

inline anvil_status run_multi(const MultiProduct& m, const Plan& plan, DeviceState* dev, cudaStream_t s, TailSumParams* rest) {
    PairMultiParams g;
    memset(&g, 0, sizeof(g));
    Product q = m.q;
    const GemmEpilogue& e2 = m.results > 1 ? m.epi2 : q.epi;
    anvil_status st = fill_pair(q, plan, dev, &g, &e2);
    if (st != ANVIL_OK) return st;
    for (int i = 1; i < m.results * m.segments; ++i)
        if ((st = encode(&g.tm_a2[i - 1], 2, q.f16, m.a[i].p, m.a[i].cols, m.a[i].rows, m.a[i].ld, 64, q.a_mn ? 64 : 128)) ||
            (st = encode(&g.tm_b2[i - 1], 2, q.f16, m.b[i].p, m.b[i].cols, m.b[i].rows, m.b[i].ld, 64, q.b_mn ? 64 : PAIR_COLS / 2)))
            return st;
    const int es = e2.out_f32 ? 4 : 2, box = g.box_bytes / es;
    if (g.out_tma && (st = encode(&g.tm_out2, es, q.f16, e2.out, q.cols, q.rows, e2.ldout, box, 128))) return st;
    if (g.in_tma && (st = encode(&g.tm_in2, es, q.f16, e2.in, q.cols, q.rows, e2.ldin, box, 128))) return st;
    g.epi2 = e2;
    g.segments = m.segments;
    g.seg_kb = static_cast<int>(ceil_div(q.k, GEMM_BK));
    g.k = static_cast<int>(multi_k(q.k, m.segments));
    g.result_tiles = g.tiles_r;
    g.tiles_r *= m.results;
    const cudaError_t e = profiled(ANVIL_KERNEL_LINEAR_PRODUCT, s, [&] { return launch_pair_multi(g, dev->sm_count, s); });
    if (e) return cuda_fail(e, "linear product launch");
    if (plan.tail) {
        fill_rest(q, plan, g, rest);
        rest->epi2 = e2;
        rest->result_tiles = g.result_tiles;
    }
    return ANVIL_OK;
}

// The finishing launch, where there is anything to finish.
inline anvil_status run_finish(const FinishParams& f, cudaStream_t s) {
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

inline Stored stored_weight(const void* w, int n, int k, int64_t ldw, bool transposed) {
    return transposed ? Stored{w, k, ldw, n} : Stored{w, n, ldw, k};
}

}  // namespace anvil
