// anvil_adamw_api.cu -- the C ABI of AdamW over many tensors (include/anvil.h): argument checks
// (before any CUDA call), the scalars of a step, and the tensors sorted into launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "../../include/anvil.h"
#include "anvil_adamw.h"
#include "anvil_host.h"
#include "anvil_types.cuh"

using namespace anvil;

static_assert(ANVIL_ADAMW_BLOCK == ADAMW_BLOCK, "ANVIL_ADAMW_BLOCK");

namespace {

bool off(const void* p, int es) { return (reinterpret_cast<uintptr_t>(p) & (es - 1)) != 0; }
int64_t blocks_of(int64_t count) { return (count + ADAMW_BLOCK - 1) / ADAMW_BLOCK; }

// The ranges of one array of every tensor (its role), in order of their addresses.
struct Role {
    Range *r, *end;
    bool written;
};
// No written range shares a byte with any other.  The arrays of a role are often neighbours in one
// buffer; otherwise a sweep over all ranges, the roles merged.
bool disjoint(Role* roles, int nroles) {
    const auto below = [](const Range& a, const Range& b) { return a.lo < b.lo; };
    bool apart = true;
    for (int i = 0; i < nroles; ++i) {
        Role& x = roles[i];
        if (!std::is_sorted(x.r, x.end, below)) std::sort(x.r, x.end, below);
        if (x.r == x.end) continue;
        uintptr_t hi = x.r->hi;
        for (const Range* q = x.r + 1; q < x.end; ++q) {
            if (x.written && q->lo < hi) return false;
            if (q->hi > hi) hi = q->hi;
        }
        for (int k = 0; k < i; ++k)
            if (roles[k].r != roles[k].end && overlap({x.r->lo, hi}, {roles[k].r->lo, (roles[k].end - 1)->hi})) apart = false;
        (x.end - 1)->hi = hi;  // (a read range may end before an earlier one)
    }
    if (apart) return true;
    uintptr_t written = 0, read = 0;  // ends of what has been passed
    uintptr_t next[8];
    for (int i = 0; i < nroles; ++i) next[i] = roles[i].r != roles[i].end ? roles[i].r->lo : UINTPTR_MAX;
    for (;;) {
        int k = 0;
        for (int i = 1; i < nroles; ++i)
            if (next[i] < next[k]) k = i;
        if (next[k] == UINTPTR_MAX) return true;
        Role& x = roles[k];
        if (x.r->lo < written || (x.written && x.r->lo < read)) return false;
        uintptr_t& end = x.written ? written : read;
        if (x.r->hi > end) end = x.r->hi;
        next[k] = ++x.r != x.end ? x.r->lo : UINTPTR_MAX;
    }
}
Range range(const void* p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p ? Range{lo, lo + static_cast<uintptr_t>(bytes)} : Range{0, 0};
}

constexpr int ROLES = 6;
template <class T, class Get>
anvil_status check_ranges(const T* tensors, int n, const bool (&written)[ROLES], Get get) {
    Range* all = new (std::nothrow) Range[static_cast<size_t>(n) * ROLES];
    if (!all) {
        set_error_text("out of host memory");
        return ANVIL_ERR_CUDA;
    }
    Role roles[ROLES];
    for (int k = 0; k < ROLES; ++k) {
        Range* to = all + static_cast<size_t>(k) * n;
        roles[k] = {to, to, written[k]};
        for (int i = 0; i < n; ++i) {
            const Range r = get(tensors[i], k);
            if (r.lo < r.hi) *roles[k].end++ = r;  // (others are absent or empty)
        }
    }
    const bool ok = disjoint(roles, ROLES);
    delete[] all;
    return ok ? ANVIL_OK : ANVIL_ERR_ALIAS;
}

int size_of(int dtype) { return dtype == ANVIL_F32 ? 4 : 2; }
// Whether a warp may take four neighbours at once of an array of es bytes a value.
bool vector(const void* p, int es) { return !(reinterpret_cast<uintptr_t>(p) & (4 * es - 1)); }

// Tensors of one kind share a launch: how param is stored, grad's type, states in 8 bits, all on vector boundaries.
int kind_of(const anvil_adamw_tensor& t) {
    const int param = t.mantissa ? ADAMW_SPLIT : t.param_dtype == ANVIL_F32 ? ADAMW_F32 : t.param_dtype == ANVIL_BF16 ? ADAMW_BF16 : ADAMW_F16;
    const int es = t.scales ? 1 : 4;
    const bool vec = vector(t.param, size_of(t.param_dtype)) && vector(t.mantissa, 2) && vector(t.grad, size_of(t.grad_dtype)) &&
                     vector(t.exp_avg, es) && vector(t.exp_avg_sq, es);
    return param << 4 | t.grad_dtype << 2 | (t.scales ? 2 : 0) | (vec ? 1 : 0);
}
constexpr int KINDS = 64;
constexpr int64_t FEW_BLOCKS = 152 * 8;  // a turn of the SMs' blocks
bool dtype_ok(int d) { return d == ANVIL_F32 || d == ANVIL_BF16 || d == ANVIL_F16; }

Range step_range(const anvil_adamw_tensor& t, int role) {
    const int es = t.scales ? 1 : 4;
    switch (role) {
        case 0: return range(t.param, t.count * size_of(t.param_dtype));
        case 1: return range(t.mantissa, t.count * 2);
        case 2: return range(t.grad, t.count * size_of(t.grad_dtype));
        case 3: return range(t.exp_avg, t.count * es);
        case 4: return range(t.exp_avg_sq, t.count * es);
        default: return range(t.scales, blocks_of(t.count) * 8);
    }
}
Range values_range(const anvil_adamw_state& t, int role) {
    switch (role) {
        case 0: return range(t.exp_avg, t.count);
        case 1: return range(t.exp_avg_sq, t.count);
        case 2: return range(t.scales, blocks_of(t.count) * 8);
        case 3: return range(t.m, t.count * 4);
        case 4: return range(t.v, t.count * 4);
        default: return {0, 0};
    }
}

// Collects tensors of one kind and launches them, ADAMW_MANY or so many chunks at a time.
template <class Launch>
struct Batches {
    AdamwGroup g;
    Launch launch;
    // blocks: of all the tensors together
    Batches(Launch f, int64_t blocks) : launch(f) {
        g.p.tensors = g.chunks = 0;
        g.p.chunk = adamw_chunk(blocks);
    }
    cudaError_t flush() {
        if (!g.p.tensors) return cudaSuccess;
        const cudaError_t e = launch(g);
        g.p.tensors = g.chunks = 0;
        return e;
    }
    cudaError_t add(AdamwTensor t) {
        const int64_t chunks = (blocks_of(t.count) + g.p.chunk - 1) / g.p.chunk;
        if (g.p.tensors == ADAMW_MANY || g.chunks + chunks > INT32_MAX) {
            const cudaError_t e = flush();
            if (e) return e;
        }
        t.chunk0 = g.chunks;
        g.chunks += static_cast<int>(chunks);
        g.p.t[g.p.tensors++] = t;
        return cudaSuccess;
    }
};

anvil_status check_config(const anvil_adamw_config* c) {
    // (a NaN fails every comparison)
    if (!c || !(c->beta1 >= 0 && c->beta1 < 1) || !(c->beta2 >= 0 && c->beta2 < 1) || !(c->eps >= 0) || !(fabs(c->lr) < 1e30) ||
        !(fabs(c->weight_decay) < 1e30) || !(fabs(c->grad_scale) < 1e30) || c->step < 1)
        return ANVIL_ERR_INVALID_ARG;
    return ANVIL_OK;
}

}  // namespace

extern "C" {

anvil_status anvil_adamw_scalars(const anvil_adamw_config* c, float* scalars) {
    const anvil_status st = check_config(c);
    if (st != ANVIL_OK || !scalars) return st != ANVIL_OK ? st : ANVIL_ERR_INVALID_ARG;
    const double t = static_cast<double>(c->step);
    scalars[0] = static_cast<float>(c->lr / (1.0 - pow(c->beta1, t)));
    scalars[1] = static_cast<float>(1.0 / sqrt(1.0 - pow(c->beta2, t)));
    scalars[2] = static_cast<float>(1.0 - c->lr * c->weight_decay);
    scalars[3] = static_cast<float>(c->grad_scale);
    return ANVIL_OK;
}

anvil_status anvil_adamw_step(const anvil_adamw_tensor* tensors, int ntensors, const anvil_adamw_config* config,
                              const float* d_scalars, void* stream) {
    float scalars[4];
    anvil_status st = anvil_adamw_scalars(config, scalars);
    if (st != ANVIL_OK) return st;
    if (ntensors < 0 || (ntensors > 0 && !tensors)) return ANVIL_ERR_INVALID_ARG;
    if (ntensors > ANVIL_MAX_TENSORS) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    if (off(d_scalars, 4)) return ANVIL_ERR_ALIGNMENT;
    uint64_t kinds = 0;  // that there are
    for (int i = 0; i < ntensors; ++i) {
        const anvil_adamw_tensor& t = tensors[i];
        if (t.count < 0 || !dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || (t.mantissa && t.param_dtype != ANVIL_BF16))
            return ANVIL_ERR_INVALID_ARG;
        if (t.param_dtype != ANVIL_F32 && t.grad_dtype != ANVIL_F32 && t.grad_dtype != t.param_dtype) return ANVIL_ERR_INVALID_ARG;
        if (t.count == 0) continue;
        if (t.count > ANVIL_MAX_COUNT) return ANVIL_ERR_UNSUPPORTED_SHAPE;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return ANVIL_ERR_INVALID_ARG;
        const int es = t.scales ? 1 : 4;
        if (off(t.param, size_of(t.param_dtype)) || off(t.mantissa, 2) || off(t.grad, size_of(t.grad_dtype)) ||
            off(t.exp_avg, es) || off(t.exp_avg_sq, es) || off(t.scales, 4))
            return ANVIL_ERR_ALIGNMENT;
        kinds |= 1ull << kind_of(t);
    }
    if (!kinds) return ANVIL_OK;
    const bool written[ROLES] = {true, true, false, true, true, true};
    if ((st = check_ranges(tensors, ntensors, written, step_range)) != ANVIL_OK) return st;
    if (d_scalars) {
        const Range s = range(d_scalars, 16);
        for (int i = 0; i < ntensors; ++i)
            for (int k = 0; k < ROLES; ++k)
                if (written[k] && tensors[i].count && overlap(s, step_range(tensors[i], k))) return ANVIL_ERR_ALIAS;
    }
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    int64_t blocks[KINDS] = {0};
    for (int i = 0; i < ntensors; ++i)
        if (tensors[i].count) blocks[kind_of(tensors[i])] += blocks_of(tensors[i].count);
    for (int kind = 0; kind < KINDS; ++kind) {
        if (!(kinds >> kind & 1)) continue;
        // a few blocks on vector boundaries go with those that are not: a launch takes longer
        const bool both = !(kind & 1) && blocks[kind | 1] <= FEW_BLOCKS;
        if ((kind & 1) && blocks[kind & ~1] && blocks[kind] <= FEW_BLOCKS) continue;
        const int param = kind >> 4, grad = kind >> 2 & 3;
        const bool codes = kind >> 1 & 1, vec = kind & 1;
        auto launch = [&](const AdamwGroup& g) {
            return profiled(ANVIL_KERNEL_ADAMW, s, [&] { return launch_adamw(g, param, grad, codes, vec, s); });
        };
        Batches<decltype(launch)> batch(launch, blocks[kind] + (both ? blocks[kind | 1] : 0));
        batch.g.p.beta1 = static_cast<float>(config->beta1);
        batch.g.p.c1 = static_cast<float>(1.0 - config->beta1);
        batch.g.p.beta2 = static_cast<float>(config->beta2);
        batch.g.p.c2 = static_cast<float>(1.0 - config->beta2);
        batch.g.p.eps = static_cast<float>(config->eps);
        for (int k = 0; k < 4; ++k) batch.g.p.scalars[k] = scalars[k];
        batch.g.p.d_scalars = d_scalars;
        for (int i = 0; i < ntensors; ++i) {
            const anvil_adamw_tensor& t = tensors[i];
            if (t.count == 0 || (both ? kind_of(t) & ~1 : kind_of(t)) != kind) continue;
            if ((e = batch.add({t.param, t.mantissa, t.grad, t.exp_avg, t.exp_avg_sq, t.scales, t.count, 0})))
                return cuda_fail(e, "AdamW launch");
        }
        if ((e = batch.flush())) return cuda_fail(e, "AdamW launch");
    }
    return ANVIL_OK;
}

anvil_status anvil_adamw_values(const anvil_adamw_state* states, int nstates, void* stream) {
    if (nstates < 0 || (nstates > 0 && !states)) return ANVIL_ERR_INVALID_ARG;
    if (nstates > ANVIL_MAX_TENSORS) return ANVIL_ERR_UNSUPPORTED_SHAPE;
    bool any = false;
    for (int i = 0; i < nstates; ++i) {
        const anvil_adamw_state& t = states[i];
        if (t.count < 0) return ANVIL_ERR_INVALID_ARG;
        if (t.count == 0) continue;
        if (t.count > ANVIL_MAX_COUNT) return ANVIL_ERR_UNSUPPORTED_SHAPE;
        if (!t.exp_avg || !t.exp_avg_sq || !t.scales || !t.m || !t.v) return ANVIL_ERR_INVALID_ARG;
        if (off(t.scales, 4) || off(t.m, 4) || off(t.v, 4)) return ANVIL_ERR_ALIGNMENT;
        any = true;
    }
    if (!any) return ANVIL_OK;
    const bool written[ROLES] = {false, false, false, true, true, false};
    anvil_status st = check_ranges(states, nstates, written, values_range);
    if (st != ANVIL_OK) return st;
    DeviceState* dev = nullptr;
    if ((st = device_setup(&dev)) != ANVIL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const auto on_vectors = [](const anvil_adamw_state& t) {
        return vector(t.exp_avg, 1) && vector(t.exp_avg_sq, 1) && vector(t.m, 4) && vector(t.v, 4);
    };
    int64_t blocks[2] = {0, 0};
    for (int i = 0; i < nstates; ++i)
        if (states[i].count) blocks[on_vectors(states[i])] += blocks_of(states[i].count);
    const bool both = blocks[0] && blocks[1] <= FEW_BLOCKS;  // as above
    for (int vec = 0; vec < (both ? 1 : 2); ++vec) {
        auto launch = [&](const AdamwGroup& g) {
            return profiled(ANVIL_KERNEL_ADAMW, s, [&] { return launch_adamw_values(g, vec != 0, s); });
        };
        Batches<decltype(launch)> batch(launch, blocks[vec] + (both ? blocks[1] : 0));
        for (int i = 0; i < nstates; ++i) {
            const anvil_adamw_state& t = states[i];
            if (t.count == 0 || (!both && on_vectors(t) != (vec != 0))) continue;
            if ((e = batch.add({t.m, nullptr, t.v, const_cast<void*>(t.exp_avg), const_cast<void*>(t.exp_avg_sq),
                                const_cast<float*>(t.scales), t.count, 0})))
                return cuda_fail(e, "AdamW launch");
        }
        if ((e = batch.flush())) return cuda_fail(e, "AdamW launch");
    }
    return ANVIL_OK;
}

}  // extern "C"
