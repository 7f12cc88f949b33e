// anvil_gated_api.cu -- the C ABI of the gated layer (include/anvil.h): argument checks (before any CUDA
// call), workspace layouts, and the choice of kernels from the sizes, types and alignment.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/anvil.h"
#include "anvil_block_host.h"

using namespace anvil;

namespace {

// The columns that plan_product sees: a tile of the pair kernel holds GATED_COLS of y.
int plan_cols(int n) { return static_cast<int>(2 * ceil_div(n, GATED_COLS) * GATED_COLS); }

// The row kernel where one tile of up to 32 tokens takes them all, or its blocks are all on SMs of their own.  Row kernel/pair
// kernel, us: 16 x 2816 x 768 6.5/8.8, 16 x 11008 x 4096 33/43, 32 x 12288 x 1024 11.7/17.4, 32 x 40000 x 2048 64.9/65.3;
// 64 x 4096 x 1024 (128 blocks) 8.3/10.1, 64 x 8192 x 4096 (256) 33.3/29, 64 x 10000 x 768 (314) 16.5/13.8.
Plan plan_forward(int64_t rows, int n, int k, bool k_major, double cycles) {
    Plan p = {};
    const int64_t tiles = ceil_div(n, ROW_TILE_A / 2);
    if (k_major && token_product(rows, plan_cols(n), k)) p.tokens = p.few = true;
    else if (rows <= ROW_TOKENS || (rows <= FEW_ROWS && tiles * row_tiles(rows) <= PLAN_SMS)) set_rows(rows, tiles, ceil_div(k, GEMM_BK), &p);
    else p = plan_product(rows, plan_cols(n), k, false, k_major, cycles, ALL_FREE);
    return p;
}

GemmEpilogue forward_epilogue(const anvil_gated_desc* d) {
    GemmEpilogue e = {};
    e.act = d->activation;
    e.z = d->preact_gate;
    e.ldz = d->ldzg;
    e.out = d->y;
    e.ldout = d->ldy;
    return e;
}

struct GatedLayout {
    Stored x, w[2];
    Plan plan;
    size_t off_x, off_w[2], off_part, total;
};
GatedLayout gated_layout(const anvil_gated_desc* d) {
    GatedLayout L;
    const bool tr = d->weight_transposed != 0;
    L.x = {d->x, d->rows, d->ldx, d->k};
    L.w[0] = stored_weight(d->gate, d->n, d->k, d->ldgate, tr);
    L.w[1] = stored_weight(d->up, d->n, d->k, d->ldup, tr);
    L.off_x = 0;
    L.off_w[0] = copy_bytes(L.x);
    L.off_w[1] = L.off_w[0] + copy_bytes(L.w[0]);
    L.off_part = L.off_w[1] + copy_bytes(L.w[1]);
    GemmEpilogue e = forward_epilogue(d);
    double cycles = epilogue_cycles(e, d->rows);
    if (d->preact_up) cycles += aligned16(d->preact_up, d->ldzu, 2, d->rows) ? 2500.0 : 12000.0;
    L.plan = plan_forward(d->rows, d->n, d->k, !tr, cycles);
    L.total = L.off_part + L.plan.part;
    return L;
}

anvil_status check_gated(const anvil_gated_desc* d) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    const anvil_status st = check_linear_sizes(d->rows, d->n, d->k, d->dtype, d->activation);
    if (st != ANVIL_OK || d->rows == 0) return st;
    if (!d->x || !d->gate || !d->up || !d->y) return ANVIL_ERR_INVALID_ARG;
    const bool tr = d->weight_transposed != 0;
    const int64_t wr = tr ? d->k : d->n, wc = tr ? d->n : d->k;
    if (bad_ld(d->rows, d->k, d->ldx) || bad_ld(wr, wc, d->ldgate) || bad_ld(wr, wc, d->ldup) || bad_ld(d->rows, d->n, d->ldy) ||
        (d->preact_gate && bad_ld(d->rows, d->n, d->ldzg)) || (d->preact_up && bad_ld(d->rows, d->n, d->ldzu)))
        return ANVIL_ERR_INVALID_ARG;
    if (misaligned(d->x, 2) || misaligned(d->gate, 2) || misaligned(d->up, 2) || misaligned(d->y, 2) ||
        misaligned(d->preact_gate, 2) || misaligned(d->preact_up, 2))
        return ANVIL_ERR_ALIGNMENT;
    return ANVIL_OK;
}

int grad_activation(const anvil_gated_grad_desc* d) { return d->activation & ~ANVIL_DZ_TWO_PARTS; }

GemmEpilogue dx_epilogue(const anvil_gated_grad_desc* d) {
    GemmEpilogue e = {};
    e.out = d->dx;
    e.ldout = d->lddx;
    return e;
}
GemmEpilogue dweight_epilogue(const anvil_gated_grad_desc* d, void* dw, int64_t ld) {
    GemmEpilogue e = {};
    e.out = dw;
    e.ldout = ld;
    e.out_f32 = d->dweight_dtype == ANVIL_F32;
    if (d->accumulate) {
        e.in = dw;
        e.ldin = ld;
    }
    return e;
}

// dz: dg and du [rows, n8] each, n8 = n rounded up to eights; in two parts dg, its rest, du, its rest.
struct GatedGradLayout {
    Stored x, w[2];
    int parts;
    int64_t n8;
    Plan pdx, pdw;
    size_t off_dz, off_x, off_w[2], off_part, total;
};
GatedGradLayout gated_grad_layout(const anvil_gated_grad_desc* d) {
    GatedGradLayout L;
    memset(&L, 0, sizeof(L));
    const bool tr = d->weight_transposed != 0;
    L.x = {d->x, d->rows, d->ldx, d->k};
    L.w[0] = stored_weight(d->gate, d->n, d->k, d->ldgate, tr);
    L.w[1] = stored_weight(d->up, d->n, d->k, d->ldup, tr);
    L.parts = d->activation & ANVIL_DZ_TWO_PARTS ? 2 : 1;
    L.n8 = (d->n + 7) & ~7;
    size_t at = align256(2 * static_cast<size_t>(d->rows) * 2 * L.parts * L.n8);
    L.off_x = at;
    if (d->dgate) at += copy_bytes(L.x);
    for (int i = 0; i < 2; ++i) {
        L.off_w[i] = at;
        if (d->dx) at += copy_bytes(L.w[i]);
    }
    L.off_part = at;
    const int64_t wr = multi_rows(tr ? d->k : d->n, 2), kdx = multi_k(d->n, 2 * L.parts), kdw = multi_k(d->rows, L.parts);
    const int wc = tr ? d->n : d->k;
    const double ex = epilogue_cycles(dx_epilogue(d), d->rows);
    const double ew = epilogue_cycles(dweight_epilogue(d, d->dgate, d->lddgate), tr ? d->k : d->n);
    if (d->dx && d->dgate) plan_both(d->rows, d->k, kdx, false, tr, ex, wr, wc, kdw, ew, &L.pdx, &L.pdw);
    else if (d->dx) L.pdx = plan_product(d->rows, d->k, kdx, false, tr, ex, ALL_FREE);
    else if (d->dgate) L.pdw = plan_product(wr, wc, kdw, false, false, ew, ALL_FREE);
    L.total = at + L.pdx.part + L.pdw.part;
    return L;
}

anvil_status check_gated_grad(const anvil_gated_grad_desc* d) {
    if (!d) return ANVIL_ERR_INVALID_ARG;
    const anvil_status st = check_linear_sizes(d->rows, d->n, d->k, d->dtype, grad_activation(d));
    if (st != ANVIL_OK) return st;
    // 32-bit numbers of the k-blocks of every segment together
    if (d->rows > ANVIL_MAX_ROWS / 4) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    if ((d->dgate != nullptr) != (d->dup != nullptr)) return ANVIL_ERR_INVALID_ARG;
    const bool tr = d->weight_transposed != 0;
    const int64_t wr = tr ? d->k : d->n, wc = tr ? d->n : d->k;
    if (d->dgate) {
        if (d->dweight_dtype != ANVIL_F32 && d->dweight_dtype != d->dtype) return ANVIL_ERR_INVALID_ARG;
        if (bad_ld(wr, wc, d->lddgate) || bad_ld(wr, wc, d->lddup)) return ANVIL_ERR_INVALID_ARG;
        if (misaligned(d->dgate, size_of(d->dweight_dtype)) || misaligned(d->dup, size_of(d->dweight_dtype)))
            return ANVIL_ERR_ALIGNMENT;
    }
    if (d->rows == 0 || (!d->dx && !d->dgate)) return ANVIL_OK;
    if (!d->dy || !d->preact_gate || !d->preact_up || (d->dgate && !d->x) || (d->dx && (!d->gate || !d->up)))
        return ANVIL_ERR_INVALID_ARG;
    if (bad_ld(d->rows, d->n, d->lddy) || bad_ld(d->rows, d->n, d->ldzg) || bad_ld(d->rows, d->n, d->ldzu) ||
        (d->dgate && bad_ld(d->rows, d->k, d->ldx)) ||
        (d->dx && (bad_ld(wr, wc, d->ldgate) || bad_ld(wr, wc, d->ldup) || bad_ld(d->rows, d->k, d->lddx))))
        return ANVIL_ERR_INVALID_ARG;
    if (misaligned(d->dy, 2) || misaligned(d->x, 2) || misaligned(d->gate, 2) || misaligned(d->up, 2) ||
        misaligned(d->preact_gate, 2) || misaligned(d->preact_up, 2) || misaligned(d->dx, 2))
        return ANVIL_ERR_ALIGNMENT;
    return ANVIL_OK;
}

anvil_status run_gated(const anvil_gated_desc* d, const GatedLayout& L, DeviceState* dev, uint8_t* ws, cudaStream_t s) {
    anvil_status st;
    cudaError_t e;
    const bool tr = d->weight_transposed != 0, f16 = d->dtype == ANVIL_F16;
    const GemmEpilogue epi = forward_epilogue(d);
    if (L.plan.tokens) {
        TokenGatedParams g;
        memset(&g, 0, sizeof(g));
        g.x = L.x.p;
        g.w = L.w[0].p;
        g.w2 = L.w[1].p;
        g.epi = epi;
        g.z2 = d->preact_up;
        g.ldz2 = d->ldzu;
        g.ldx = L.x.ld;
        g.ldw = L.w[0].ld;
        g.ldw2 = L.w[1].ld;
        g.rows = static_cast<int>(d->rows);
        g.cols = d->n;
        g.k = d->k;
        g.f16 = f16;
        e = profiled(ANVIL_KERNEL_GATED_PRODUCT, s, [&] { return launch_tokens_gated(g, s); });
        return e ? cuda_fail(e, "gated product launch") : ANVIL_OK;
    }
    if (L.plan.few) {
        RowGatedParams g;
        memset(&g, 0, sizeof(g));
        if ((st = encode(&g.tm_a, 2, f16, L.w[0].p, L.w[0].cols, L.w[0].rows, L.w[0].ld, 64, 64)) ||
            (st = encode(&g.tm_a2, 2, f16, L.w[1].p, L.w[1].cols, L.w[1].rows, L.w[1].ld, 64, 64)) ||
            (st = encode(&g.tm_b, 2, f16, L.x.p, L.x.cols, L.x.rows, L.x.ld, 64, L.plan.bn)))
            return st;
        g.epi = epi;
        g.z2 = d->preact_up;
        g.ldz2 = d->ldzu;
        g.na = d->n;
        g.nb = static_cast<int>(d->rows);
        g.k = d->k;
        g.a_mn = tr;
        g.f16 = f16;
        g.splits = L.plan.splits;
        g.kb_per_split = L.plan.kb;
        g.err = dev->err;
        e = profiled(ANVIL_KERNEL_GATED_PRODUCT, s, [&] { return launch_row_gated(g, L.plan.bn, dev->sm_count, s); });
        return e ? cuda_fail(e, "gated product launch") : ANVIL_OK;
    }
    PairGatedParams g;
    memset(&g, 0, sizeof(g));
    if ((st = encode(&g.tm_a, 2, f16, L.x.p, L.x.cols, L.x.rows, L.x.ld, 64, 128)) ||
        (st = encode(&g.tm_b, 2, f16, L.w[0].p, L.w[0].cols, L.w[0].rows, L.w[0].ld, 64, tr ? 64 : GATED_COLS)) ||
        (st = encode(&g.tm_b2, 2, f16, L.w[1].p, L.w[1].cols, L.w[1].rows, L.w[1].ld, 64, tr ? 64 : GATED_COLS)))
        return st;
    g.epi = epi;
    g.z2 = d->preact_up;
    g.ldz2 = d->ldzu;
    g.rows = static_cast<int>(d->rows);
    g.cols = d->n;
    g.k = d->k;
    g.b_mn = tr;
    g.f16 = f16;
    g.out_tma = aligned16(d->y, d->ldy, 2, d->rows);
    g.z_tma = d->preact_gate && aligned16(d->preact_gate, d->ldzg, 2, d->rows);
    g.z2_tma = d->preact_up && aligned16(d->preact_up, d->ldzu, 2, d->rows);
    g.box_bytes = 64;
    if (g.out_tma && (st = encode(&g.tm_out, 2, f16, d->y, d->n, d->rows, d->ldy, 32, 128))) return st;
    if (g.z_tma && (st = encode(&g.tm_z, 2, f16, d->preact_gate, d->n, d->rows, d->ldzg, 32, 128))) return st;
    if (g.z2_tma && (st = encode(&g.tm_z2, 2, f16, d->preact_up, d->n, d->rows, d->ldzu, 32, 128))) return st;
    float* part = reinterpret_cast<float*>(ws + L.off_part);
    if (L.plan.tail &&
        (st = encode(&g.tm_part, 4, false, part, PAIR_COLS, static_cast<int64_t>(L.plan.part / (4 * PAIR_COLS)), PAIR_COLS, 16, 128)))
        return st;
    g.tiles_r = static_cast<int>(ceil_div(d->rows, PAIR_ROWS));
    g.tiles_c = static_cast<int>(ceil_div(d->n, GATED_COLS));
    g.split = L.plan.split;
    g.units = L.plan.units;
    g.err = dev->err;
    if ((e = profiled(ANVIL_KERNEL_GATED_PRODUCT, s, [&] { return launch_pair_gated(g, dev->sm_count, s); })))
        return cuda_fail(e, "gated product launch");
    if (!L.plan.tail) return ANVIL_OK;
    const GatedTailParams f = {epi, d->preact_up, d->ldzu, part, g.rows, g.cols, g.tiles_r, g.tiles_c, L.plan.tail, f16, L.plan.split};
    e = profiled(ANVIL_KERNEL_GATED_SUM, s, [&] { return launch_gated_finish(f, s); });
    return e ? cuda_fail(e, "gated sum launch") : ANVIL_OK;
}

}  // namespace

extern "C" {

size_t anvil_gated_linear_workspace_bytes(const anvil_gated_desc* d) {
    if (check_gated(d) != ANVIL_OK || d->rows == 0) return 0;
    return gated_layout(d).total;
}

anvil_status anvil_gated_linear_forward(const anvil_gated_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
    anvil_status st = check_gated(d);
    if (st != ANVIL_OK || d->rows == 0) return st;
    const bool tr = d->weight_transposed != 0;
    const int64_t wr = tr ? d->k : d->n, wc = tr ? d->n : d->k;
    const Area a[6] = {area(d->x, d->rows, d->k, d->ldx, 2, false),       area(d->gate, wr, wc, d->ldgate, 2, false),
                       area(d->up, wr, wc, d->ldup, 2, false),             area(d->y, d->rows, d->n, d->ldy, 2, true),
                       area(d->preact_gate, d->rows, d->n, d->ldzg, 2, true), area(d->preact_up, d->rows, d->n, d->ldzu, 2, true)};
    if ((st = check_areas(a, 6, nullptr, 0)) != ANVIL_OK) return st;
    GatedLayout L = gated_layout(d);
    if ((st = check_workspace(workspace, workspace_bytes, L.total, a, 6)) != ANVIL_OK) return st;
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Copies copies = {};
    copies.add(&L.x, ws + L.off_x);
    for (int i = 0; i < 2; ++i) copies.add(&L.w[i], ws + L.off_w[i]);
    if ((st = copies.run(s)) != ANVIL_OK) return st;
    return run_gated(d, L, dev, ws, s);
}

size_t anvil_gated_linear_backward_workspace_bytes(const anvil_gated_grad_desc* d) {
    if (check_gated_grad(d) != ANVIL_OK || d->rows == 0 || (!d->dx && !d->dgate)) return 0;
    return gated_grad_layout(d).total;
}

anvil_status anvil_gated_linear_backward(const anvil_gated_grad_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
    anvil_status st = check_gated_grad(d);
    if (st != ANVIL_OK) return st;
    if (!d->dx && !d->dgate) return ANVIL_OK;
    const bool tr = d->weight_transposed != 0, f16 = d->dtype == ANVIL_F16;
    const int dws = size_of(d->dweight_dtype);
    const int64_t wr = tr ? d->k : d->n, wc = tr ? d->n : d->k;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    DeviceState* dev = nullptr;
    if (d->rows == 0) {
        if (d->accumulate || !d->dgate) return ANVIL_OK;
        if (share(area(d->dgate, wr, wc, d->lddgate, dws, true), area(d->dup, wr, wc, d->lddup, dws, true))) return ANVIL_ERR_ALIAS;
        if ((st = device_setup(&dev)) != ANVIL_OK) return st;
        if ((e = cudaMemset2DAsync(d->dgate, (wr > 1 ? d->lddgate : wc) * dws, 0, wc * dws, wr, s)) ||
            (e = cudaMemset2DAsync(d->dup, (wr > 1 ? d->lddup : wc) * dws, 0, wc * dws, wr, s)))
            return cuda_fail(e, "cudaMemset2DAsync");
        return ANVIL_OK;
    }
    const Area a[9] = {area(d->dy, d->rows, d->n, d->lddy, 2, false),
                       area(d->dgate ? d->x : nullptr, d->rows, d->k, d->ldx, 2, false),
                       area(d->dx ? d->gate : nullptr, wr, wc, d->ldgate, 2, false),
                       area(d->dx ? d->up : nullptr, wr, wc, d->ldup, 2, false),
                       area(d->preact_gate, d->rows, d->n, d->ldzg, 2, false),
                       area(d->preact_up, d->rows, d->n, d->ldzu, 2, false),
                       area(d->dx, d->rows, d->k, d->lddx, 2, true),
                       area(d->dgate, wr, wc, d->lddgate, dws, true),
                       area(d->dup, wr, wc, d->lddup, dws, true)};
    if ((st = check_areas(a, 9, nullptr, 0)) != ANVIL_OK) return st;
    GatedGradLayout L = gated_grad_layout(d);
    if ((st = check_workspace(workspace, workspace_bytes, L.total, a, 9)) != ANVIL_OK) return st;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    GatedGradParams p;
    memset(&p, 0, sizeof(p));
    p.dy = d->dy;
    p.g = d->preact_gate;
    p.u = d->preact_up;
    p.dz = ws + L.off_dz;
    p.two_parts = L.parts == 2;
    p.rows = d->rows;
    p.lddy = d->lddy;
    p.ldg = d->ldzg;
    p.ldu = d->ldzu;
    p.ldd = L.n8;
    p.cols = d->n;
    p.act = grad_activation(d);
    p.f16 = f16;
    if ((e = profiled(ANVIL_KERNEL_GATED_PREPARE, s, [&] { return launch_gated_grad(p, s); })))
        return cuda_fail(e, "gated gradient launch");
    Copies copies = {};
    if (d->dgate) copies.add(&L.x, ws + L.off_x);
    if (d->dx)
        for (int i = 0; i < 2; ++i) copies.add(&L.w[i], ws + L.off_w[i]);
    if ((st = copies.run(s)) != ANVIL_OK) return st;
    Stored dz[4];  // in the order they are stored: dg (, its rest), du (, its rest)
    for (int i = 0; i < 2 * L.parts; ++i)
        dz[i] = {ws + L.off_dz + static_cast<size_t>(i) * 2 * d->rows * L.n8, d->rows, L.n8, d->n};
    FinishParams f;
    memset(&f, 0, sizeof(f));
    f.f16 = f16;
    const bool overlap = d->dx && d->dgate;
    if (d->dx) {
        MultiProduct m;
        memset(&m, 0, sizeof(m));
        for (int i = 0; i < 2 * L.parts; ++i) {
            m.a[i] = dz[i];
            m.b[i] = L.w[i / L.parts];
        }
        m.results = 1;
        m.segments = 2 * L.parts;
        m.q.a = m.a[0];
        m.q.b = m.b[0];
        m.q.b_mn = !tr;
        m.q.rows = d->rows;
        m.q.cols = d->k;
        m.q.k = d->n;
        m.q.f16 = f16;
        m.q.epi = dx_epilogue(d);
        m.q.part = reinterpret_cast<float*>(ws + L.off_part);
        m.q.overlap_next = overlap;
        if ((st = run_multi(m, L.pdx, dev, s, &f.tail[0])) != ANVIL_OK) return st;
    }
    if (d->dgate) {
        MultiProduct m;
        memset(&m, 0, sizeof(m));
        for (int i = 0; i < 2 * L.parts; ++i) {
            m.a[i] = tr ? L.x : dz[i];
            m.b[i] = tr ? dz[i] : L.x;
        }
        m.results = 2;
        m.segments = L.parts;
        m.q.a = m.a[0];
        m.q.b = m.b[0];
        m.q.a_mn = m.q.b_mn = true;
        m.q.rows = wr;
        m.q.cols = static_cast<int>(wc);
        m.q.k = d->rows;
        m.q.f16 = f16;
        m.q.epi = dweight_epilogue(d, d->dgate, d->lddgate);
        m.epi2 = dweight_epilogue(d, d->dup, d->lddup);
        m.q.part = reinterpret_cast<float*>(ws + L.off_part + L.pdx.part);
        m.q.overlap_previous = overlap;
        if ((st = run_multi(m, L.pdw, dev, s, &f.tail[1])) != ANVIL_OK) return st;
    }
    return run_finish(f, s);
}

}  // extern "C"
