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
#include "anvil_block_host.h"
#include "anvil_logprob.h"
#include "anvil_norm.h"

using namespace anvil;

static_assert(ANVIL_ACT_SILU == ACT_SILU && ANVIL_ACT_RELU2 == ACT_RELU2, "activation codes of include/anvil.h");
static_assert(ANVIL_MAX_TOP == LOGPROB_MAX_TOP, "ANVIL_MAX_TOP");
static_assert(ANVIL_DZ_TWO_PARTS >= ACT_COUNT, "a bit of its own beside the activation codes");

namespace {

// ---------------------------------------------------------------- layer norm
anvil_status check_norm_sizes(int64_t rows, int width, int dtype, int weight_dtype) {
    if (rows < 0 || width < 1 || !valid_dtype(dtype)) return ANVIL_ERR_INVALID_ARG;
    if (weight_dtype != ANVIL_F32 && weight_dtype != dtype) return ANVIL_ERR_INVALID_ARG;
    if (rows > ANVIL_MAX_ROWS || width > ANVIL_MAX_WIDTH) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    return ANVIL_OK;
}

size_t norm_bwd_bytes(const anvil_layernorm_grad_desc* d) {
    if (d->rows == 0 || (!d->dweight && !d->dbias)) return 0;
    const int blocks = norm_bwd_max_blocks(d->rows, d->width, d->dtype);
    return blocks > 1 ? align256(sizeof(float) * 2 * static_cast<size_t>(blocks) * d->width) : 0;
}

// ---------------------------------------------------------------- the linear layer
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
    if (d->dx && d->dweight) plan_both(d->rows, d->k, L.kdx, true, tr, ex, wr, wc, L.kdw, ew, &L.pdx, &L.pdw);
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
