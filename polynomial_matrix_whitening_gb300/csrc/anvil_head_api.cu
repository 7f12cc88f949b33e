// anvil_head_api.cu -- the C ABI of the head's cross entropy (include/anvil.h): argument checks (before
// any CUDA call), workspace layouts, the pieces of the vocabulary and their products.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/anvil.h"
#include "anvil_block_host.h"

using namespace anvil;

namespace {

anvil_status check_sizes(int64_t rows, int vocab, int k, int dtype) {
    if (rows < 0 || vocab < 1 || k < 1 || (dtype != ANVIL_BF16 && dtype != ANVIL_F16)) return ANVIL_ERR_INVALID_ARG;
    if (rows > ANVIL_MAX_ROWS || vocab > ANVIL_MAX_VOCAB || k > ANVIL_MAX_FEATURES) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    const int64_t t = ceil_div(rows, 128);
    if (t * ceil_div(vocab, 128) >= (1ll << 30) || t * ceil_div(k, 128) >= (1ll << 30)) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    return ANVIL_OK;
}

// Forward: copies of unaligned operands, the statistics [parts][rows], the targets' logits [rows].
struct HeadLayout {
    Stored x, w;
    Plan plan;
    int parts;
    size_t off_x, off_w, off_stats, off_hit, total;
};
HeadLayout head_layout(const anvil_head_desc* d) {
    HeadLayout L;
    L.x = {d->x, d->rows, d->ldx, d->k};
    L.w = stored_weight(d->weight, d->vocab, d->k, d->ldw, d->weight_transposed != 0);
    memset(&L.plan, 0, sizeof(L.plan));
    // One or two rows and a weight stored by rows for which the row kernel would have a block an SM at
    // most: read without tensor cores.  The row kernel up to one tile of tokens (us, row kernel/pair kernel: 32 rows
    // 50304 x 768 21.4/25.3, 8000 x 4096 18.2/24.9, 128000 x 4096 176/172; 64 rows 20000 x 768 14.5/15.7, 32000 x
    // 4096 67/52, 5000 x 768 10.1/9.9).
    L.plan.tokens = d->rows <= HEAD_TOKENS && !d->weight_transposed && d->rows * d->k <= HEAD_TOKEN_VALUES &&
                    ceil_div(d->vocab, ROW_TILE_A) <= PLAN_SMS;
    if (!L.plan.tokens && d->rows <= ROW_TOKENS) set_rows(d->rows, ceil_div(d->vocab, ROW_TILE_A), ceil_div(d->k, GEMM_BK), &L.plan);
    if (L.plan.tokens) L.parts = head_token_blocks(d->vocab);
    else L.parts = static_cast<int>(L.plan.few ? ceil_div(d->vocab, ROW_TILE_A) : ceil_div(d->vocab, PAIR_COLS) * (PAIR_COLS / HEAD_STATS_COLS));
    L.off_x = 0;
    L.off_w = L.off_x + copy_bytes(L.x);
    L.off_stats = L.off_w + copy_bytes(L.w);
    L.off_hit = L.off_stats + align256(sizeof(float2) * static_cast<size_t>(L.parts) * d->rows);
    L.total = L.off_hit + (d->loss ? align256(sizeof(float) * d->rows) : 0);
    return L;
}

anvil_status check_head(const anvil_head_desc* d) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    const anvil_status st = check_sizes(d->rows, d->vocab, d->k, d->dtype);
    if (st != ANVIL_OK || d->rows == 0 || (!d->loss && !d->lse)) return st;
    const bool tr = d->weight_transposed != 0;
    if (!d->x || !d->weight || (d->loss && !d->targets) || bad_ld(d->rows, d->k, d->ldx) ||
        bad_ld(tr ? d->k : d->vocab, tr ? d->vocab : d->k, d->ldw))
        return ANVIL_ERR_INVALID_ARG;
    if (misaligned(d->x, 2) || misaligned(d->weight, 2) || misaligned(d->targets, d->targets_int64 ? 8 : 4) ||
        misaligned(d->loss, 4) || misaligned(d->lse, 4))
        return ANVIL_ERR_ALIGNMENT;
    return ANVIL_OK;
}

// The gradient's pieces: as many columns of the vocabulary as d takes 512 MB for, whole tiles, all but the
// last of one size.  (us, pieces of 128 MB, 256 MB, 512 MB, 1 GB, 2 GB: 8192 x 50304 x 768 1300, 1170, 1125, 1110,
// 1110; 16384 x 50304 x 768 2740, 2410, 2410, 2320, 2230; 32768 x 32000 x 1024 4530, 4150, 3880, 3870, 3720; 4096 x
// 65536 x 2048 2020, 1990, 1935, 1945, 1920; 2048 x 131072 x 4096 3855, 3730, 3855, 3725, 3675; 16384 x 131072 x 512
// 5235, 4670, 4470, 4150, 4150: four times the memory would give 8% at most.)
constexpr int64_t PIECE_BYTES = 512ll << 20;
struct HeadGradLayout {
    Stored x, w;
    int pieces, piece, last;    // columns of a piece, of the last one
    int64_t ldd, k8;            // of d, of dx's sum
    Plan pdx[2], pdw[2];        // of a whole piece and of the last one
    size_t off_scale, off_x, off_w, off_d, off_sum, off_part, part_dx, total;
};

GemmEpilogue dx_epilogue(const anvil_head_grad_desc* d, const HeadGradLayout& L, float* sum, bool first) {
    GemmEpilogue e = {};
    if (L.pieces == 1) {
        e.out = d->dx;
        e.ldout = d->lddx;
        return e;
    }
    e.out = sum;
    e.ldout = L.k8;
    e.out_f32 = 1;
    if (!first) {
        e.in = sum;
        e.ldin = L.k8;
    }
    return e;
}
GemmEpilogue dweight_epilogue(const anvil_head_grad_desc* d, int64_t first) {
    GemmEpilogue e = {};
    e.out = static_cast<uint8_t*>(d->dweight) + size_of(d->dweight_dtype) * (d->weight_transposed ? first : first * d->lddw);
    e.ldout = d->lddw;
    e.out_f32 = d->dweight_dtype == ANVIL_F32;
    if (d->accumulate) {
        e.in = e.out;
        e.ldin = d->lddw;
    }
    return e;
}

HeadGradLayout head_grad_layout(const anvil_head_grad_desc* d) {
    HeadGradLayout L;
    memset(&L, 0, sizeof(L));
    const bool tr = d->weight_transposed != 0;
    L.x = {d->x, d->rows, d->ldx, d->k};
    L.w = stored_weight(d->weight, d->vocab, d->k, d->ldw, tr);
    int64_t most = PIECE_BYTES / (2 * d->rows) / PAIR_COLS * PAIR_COLS;
    if (most < PAIR_COLS) most = PAIR_COLS;
    L.pieces = static_cast<int>(ceil_div(d->vocab, most));
    L.piece = static_cast<int>(ceil_div(ceil_div(d->vocab, L.pieces), PAIR_COLS) * PAIR_COLS);
    L.pieces = static_cast<int>(ceil_div(d->vocab, L.piece));
    L.last = d->vocab - (L.pieces - 1) * L.piece;
    L.ldd = L.pieces > 1 ? L.piece : (d->vocab + 7) & ~7;
    L.k8 = (d->k + 7) & ~7;
    size_t at = 0;
    L.off_scale = at;
    at += 256;
    L.off_x = at;
    at += copy_bytes(L.x);
    L.off_w = at;
    at += copy_bytes(L.w);
    L.off_d = at;
    at += align256(2 * static_cast<size_t>(d->rows) * L.ldd);
    L.off_sum = at;
    if (d->dx && L.pieces > 1) at += align256(sizeof(float) * static_cast<size_t>(d->rows) * L.k8);
    L.off_part = at;
    size_t part_dw = 0;
    float* aligned = reinterpret_cast<float*>(static_cast<uintptr_t>(256));  // where the sum will be, as far as costs go
    for (int i = 0; i < 2; ++i) {
        const int cols = i ? L.last : L.piece;
        const int64_t wr = tr ? d->k : cols;
        const int wc = tr ? cols : d->k;
        const double ex = epilogue_cycles(dx_epilogue(d, L, aligned, false), d->rows);
        const double ew = d->dweight ? epilogue_cycles(dweight_epilogue(d, 0), wr) : 0.0;
        if (d->dx && d->dweight) plan_both(d->rows, d->k, cols, false, tr, ex, wr, wc, d->rows, ew, &L.pdx[i], &L.pdw[i]);
        else if (d->dx) L.pdx[i] = plan_product(d->rows, d->k, cols, false, tr, ex, ALL_FREE);
        else L.pdw[i] = plan_product(wr, wc, d->rows, false, false, ew, ALL_FREE);
        if (L.pdx[i].part > L.part_dx) L.part_dx = L.pdx[i].part;
        if (L.pdw[i].part > part_dw) part_dw = L.pdw[i].part;
    }
    L.total = at + L.part_dx + part_dw;
    return L;
}

anvil_status check_head_grad(const anvil_head_grad_desc* d) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    const anvil_status st = check_sizes(d->rows, d->vocab, d->k, d->dtype);
    if (st != ANVIL_OK) return st;
    const bool tr = d->weight_transposed != 0;
    const int64_t wr = tr ? d->k : d->vocab, wc = tr ? d->vocab : d->k;
    if (d->dweight) {
        if (d->dweight_dtype != ANVIL_F32 && d->dweight_dtype != d->dtype) return ANVIL_ERR_INVALID_ARG;
        if (bad_ld(wr, wc, d->lddw)) return ANVIL_ERR_INVALID_ARG;
        if (misaligned(d->dweight, size_of(d->dweight_dtype))) return ANVIL_ERR_ALIGNMENT;
    }
    if (d->rows == 0 || (!d->dx && !d->dweight)) return ANVIL_OK;
    if (!d->x || !d->weight || !d->targets || !d->lse || !d->grad_loss || bad_ld(d->rows, d->k, d->ldx) || bad_ld(wr, wc, d->ldw) ||
        (d->dx && bad_ld(d->rows, d->k, d->lddx)))
        return ANVIL_ERR_INVALID_ARG;
    if (misaligned(d->x, 2) || misaligned(d->weight, 2) || misaligned(d->targets, d->targets_int64 ? 8 : 4) ||
        misaligned(d->lse, 4) || misaligned(d->grad_loss, 4) || misaligned(d->dx, 2))
        return ANVIL_ERR_ALIGNMENT;
    return ANVIL_OK;
}

// The product x W^T over `cols` columns of the vocabulary from `first` on, for either epilogue.
anvil_status fill_logits(const Stored& x, const Stored& w, bool tr, int64_t first, int cols, bool f16, DeviceState* dev, PairHeadParams* g) {
    Stored piece = w;
    piece.p = static_cast<const uint8_t*>(w.p) + 2 * (tr ? first : first * w.ld);
    if (tr) piece.cols = cols;
    else piece.rows = cols;
    Plan plan;
    set_whole(tiles_of(x.rows, cols), 0.0, &plan);
    anvil_status st;
    if ((st = encode(&g->tm_a, 2, f16, x.p, x.cols, x.rows, x.ld, 64, 128)) ||
        (st = encode(&g->tm_b, 2, f16, piece.p, piece.cols, piece.rows, piece.ld, 64, tr ? 64 : PAIR_COLS / 2)))
        return st;
    g->rows = static_cast<int>(x.rows);
    g->cols = cols;
    g->k = x.cols;
    g->b_mn = tr;
    g->f16 = f16;
    g->tiles_r = static_cast<int>(ceil_div(x.rows, PAIR_ROWS));
    g->tiles_c = static_cast<int>(ceil_div(cols, PAIR_COLS));
    g->split = plan.split;
    g->units = plan.units;
    g->box_bytes = 64;
    g->err = dev->err;
    g->first = static_cast<int>(first);
    return ANVIL_OK;
}

}  // namespace

extern "C" {

size_t anvil_linear_cross_entropy_workspace_bytes(const anvil_head_desc* d) {
    if (check_head(d) != ANVIL_OK || d->rows == 0 || (!d->loss && !d->lse)) return 0;
    return head_layout(d).total;
}

anvil_status anvil_linear_cross_entropy(const anvil_head_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
    anvil_status st = check_head(d);
    if (st != ANVIL_OK || d->rows == 0 || (!d->loss && !d->lse)) return st;
    const bool tr = d->weight_transposed != 0, f16 = d->dtype == ANVIL_F16;
    const int ts = d->targets_int64 ? 8 : 4;
    const Area a[5] = {area(d->x, d->rows, d->k, d->ldx, 2, false),
                       area(d->weight, tr ? d->k : d->vocab, tr ? d->vocab : d->k, d->ldw, 2, false),
                       area(d->loss ? d->targets : nullptr, 1, d->rows, 0, ts, false), area(d->loss, 1, d->rows, 0, 4, true),
                       area(d->lse, 1, d->rows, 0, 4, true)};
    if ((st = check_areas(a, 5, nullptr, 0)) != ANVIL_OK) return st;
    HeadLayout L = head_layout(d);
    if ((st = check_workspace(workspace, workspace_bytes, L.total, a, 5)) != ANVIL_OK) return st;
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaError_t e;
    Copies copies = {};
    copies.add(&L.x, ws + L.off_x);
    copies.add(&L.w, ws + L.off_w);
    if ((st = copies.run(s)) != ANVIL_OK) return st;
    const int target64 = d->targets_int64 != 0;
    float2* stats = reinterpret_cast<float2*>(ws + L.off_stats);
    float* hit = d->loss ? reinterpret_cast<float*>(ws + L.off_hit) : nullptr;
    if (L.plan.tokens) {
        const TokenHeadParams g = {L.x.p, L.w.p, L.x.ld, L.w.ld, static_cast<int>(d->rows), d->vocab, d->k, f16, d->targets, target64, stats, hit};
        e = profiled(ANVIL_KERNEL_HEAD_PRODUCT, s, [&] { return launch_head_tokens(g, s); });
    } else if (L.plan.few) {
        RowHeadParams g;
        memset(&g, 0, sizeof(g));
        if ((st = encode(&g.tm_a, 2, f16, L.w.p, L.w.cols, L.w.rows, L.w.ld, 64, tr ? 64 : ROW_TILE_A)) ||
            (st = encode(&g.tm_b, 2, f16, L.x.p, L.x.cols, L.x.rows, L.x.ld, 64, L.plan.bn)))
            return st;
        g.na = d->vocab;
        g.nb = static_cast<int>(d->rows);
        g.k = d->k;
        g.a_mn = tr;
        g.f16 = f16;
        g.splits = L.plan.splits;
        g.kb_per_split = L.plan.kb;
        g.err = dev->err;
        g.targets = d->targets;
        g.target64 = target64;
        g.stats = stats;
        g.hit = hit;
        e = profiled(ANVIL_KERNEL_HEAD_PRODUCT, s, [&] { return launch_head_rows(g, L.plan.bn, dev->sm_count, s); });
    } else {
        PairHeadParams g;
        memset(&g, 0, sizeof(g));
        if ((st = fill_logits(L.x, L.w, tr, 0, d->vocab, f16, dev, &g)) != ANVIL_OK) return st;
        g.targets = d->targets;
        g.target64 = target64;
        g.stats = stats;
        g.hit = hit;
        e = profiled(ANVIL_KERNEL_HEAD_PRODUCT, s, [&] { return launch_head_stats(g, dev->sm_count, s); });
    }
    if (e) return cuda_fail(e, "cross entropy launch");
    const HeadJoinParams j = {stats, hit, d->targets, d->loss, d->lse, d->rows, L.parts, d->vocab, target64};
    e = profiled(ANVIL_KERNEL_HEAD_SUM, s, [&] { return launch_head_join(j, s); });
    return e ? cuda_fail(e, "cross entropy launch") : ANVIL_OK;
}

size_t anvil_linear_cross_entropy_backward_workspace_bytes(const anvil_head_grad_desc* d) {
    if (check_head_grad(d) != ANVIL_OK || d->rows == 0 || (!d->dx && !d->dweight)) return 0;
    return head_grad_layout(d).total;
}

anvil_status anvil_linear_cross_entropy_backward(const anvil_head_grad_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
    anvil_status st = check_head_grad(d);
    if (st != ANVIL_OK) return st;
    if (!d->dx && !d->dweight) return ANVIL_OK;
    const bool tr = d->weight_transposed != 0, f16 = d->dtype == ANVIL_F16;
    const int64_t wr = tr ? d->k : d->vocab, wc = tr ? d->vocab : d->k;
    const int dws = size_of(d->dweight_dtype), ts = d->targets_int64 ? 8 : 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    DeviceState* dev = nullptr;
    if (d->rows == 0) {
        if (d->accumulate || !d->dweight) return ANVIL_OK;
        if ((st = device_setup(&dev)) != ANVIL_OK) return st;
        if ((e = cudaMemset2DAsync(d->dweight, (wr > 1 ? d->lddw : wc) * dws, 0, wc * dws, wr, s)))
            return cuda_fail(e, "cudaMemset2DAsync");
        return ANVIL_OK;
    }
    const Area a[7] = {area(d->x, d->rows, d->k, d->ldx, 2, false), area(d->weight, wr, wc, d->ldw, 2, false),
                       area(d->targets, 1, d->rows, 0, ts, false),  area(d->lse, 1, d->rows, 0, 4, false),
                       area(d->grad_loss, 1, d->rows, 0, 4, false), area(d->dx, d->rows, d->k, d->lddx, 2, true),
                       area(d->dweight, wr, wc, d->lddw, dws, true)};
    if ((st = check_areas(a, 7, nullptr, 0)) != ANVIL_OK) return st;
    HeadGradLayout L = head_grad_layout(d);
    if ((st = check_workspace(workspace, workspace_bytes, L.total, a, 7)) != ANVIL_OK) return st;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int target64 = d->targets_int64 != 0;
    float* scale = reinterpret_cast<float*>(ws + L.off_scale);
    float* sum = reinterpret_cast<float*>(ws + L.off_sum);
    const HeadScaleParams unit = {d->grad_loss, d->targets, scale, d->rows, target64, f16};
    if ((e = profiled(ANVIL_KERNEL_HEAD_PREPARE, s, [&] { return launch_head_scale(unit, s); })))
        return cuda_fail(e, "cross entropy gradient launch");
    Copies copies = {};
    copies.add(&L.x, ws + L.off_x);
    copies.add(&L.w, ws + L.off_w);
    if ((st = copies.run(s)) != ANVIL_OK) return st;
    for (int i = 0; i < L.pieces; ++i) {
        const bool last = i == L.pieces - 1;
        const int64_t first = static_cast<int64_t>(i) * L.piece;
        const int cols = last ? L.last : L.piece;
        PairHeadParams g;
        memset(&g, 0, sizeof(g));
        if ((st = fill_logits(L.x, L.w, tr, first, cols, f16, dev, &g)) != ANVIL_OK) return st;
        g.targets = d->targets;
        g.target64 = target64;
        g.lse = d->lse;
        g.grad = d->grad_loss;
        g.scale = scale;
        g.epi.out = ws + L.off_d;
        g.epi.ldout = L.ldd;
        if ((st = encode(&g.tm_out, 2, f16, g.epi.out, (cols + 7) & ~7, d->rows, L.ldd, 32, 128))) return st;
        if ((e = profiled(ANVIL_KERNEL_HEAD_PRODUCT, s, [&] { return launch_head_dlogits(g, dev->sm_count, s); })))
            return cuda_fail(e, "cross entropy gradient launch");
        const Stored dz = {ws + L.off_d, d->rows, L.ldd, cols};
        FinishParams f;
        memset(&f, 0, sizeof(f));
        f.f16 = f16;
        const Plan &pdx = L.pdx[last], &pdw = L.pdw[last];
        const bool overlap = d->dx && d->dweight;
        MultiProduct m;
        if (d->dx) {
            memset(&m, 0, sizeof(m));
            m.results = m.segments = 1;
            m.q.a = dz;
            m.q.b = L.w;
            m.q.b.p = static_cast<const uint8_t*>(L.w.p) + 2 * (tr ? first : first * L.w.ld);
            if (tr) m.q.b.cols = cols;
            else m.q.b.rows = cols;
            m.q.b_mn = !tr;
            m.q.rows = d->rows;
            m.q.cols = d->k;
            m.q.k = cols;
            m.q.f16 = f16;
            m.q.epi = dx_epilogue(d, L, sum, i == 0);
            m.q.part = reinterpret_cast<float*>(ws + L.off_part);
            m.q.overlap_next = overlap;
            if (L.pieces == 1) {
                m.q.epi.scale = scale + 1;
                st = run_multi(m, pdx, dev, s, &f.tail[0]);
            } else {
                m.q.one_chain = true;
                st = run_product(m.q, pdx, dev, s, &f.tail[0]);
            }
            if (st != ANVIL_OK) return st;
        }
        if (d->dweight) {
            memset(&m, 0, sizeof(m));
            m.results = m.segments = 1;
            m.q.a = tr ? L.x : dz;
            m.q.b = tr ? dz : L.x;
            m.q.a_mn = m.q.b_mn = true;
            m.q.rows = tr ? d->k : cols;
            m.q.cols = tr ? cols : d->k;
            m.q.k = d->rows;
            m.q.f16 = f16;
            m.q.epi = dweight_epilogue(d, first);
            m.q.part = reinterpret_cast<float*>(ws + L.off_part + L.part_dx);
            m.q.overlap_previous = overlap;
            m.q.epi.scale = scale + 1;
            if ((st = run_multi(m, pdw, dev, s, &f.tail[1])) != ANVIL_OK) return st;
        }
        if ((st = run_finish(f, s)) != ANVIL_OK) return st;
    }
    if (!d->dx || L.pieces == 1) return ANVIL_OK;
    const HeadRoundParams p = {sum, d->dx, scale + 1, d->rows, d->rows > 1 ? d->lddx : d->k, d->k, f16};
    e = profiled(ANVIL_KERNEL_HEAD_SUM, s, [&] { return launch_head_round(p, s); });
    return e ? cuda_fail(e, "cross entropy gradient launch") : ANVIL_OK;
}

}  // extern "C"
