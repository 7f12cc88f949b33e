// anvil_norm.cu -- layer norm, forward and backward, for sm_103a.
//
//   forward   mean = sum_j x_j / n,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / n + eps),
//             y_j = (x_j - mean) rstd w_j + b_j
//   backward  h_j = (x_j - mean) rstd,  g_j = dy_j w_j,
//             dx_j = rstd (g_j - mean_j(g) - h_j mean_j(g h)) [+ r_j],
//             dw_j = sum over rows of dy_j h_j,  db_j = sum over rows of dy_j
//
// Both passes read each input once and write each output once, so HBM bounds them.  A row
// belongs to a team of threads that keeps it in registers between the reductions and the
// store (the variance is taken from the centred values, in a second pass over registers,
// not from a difference of large sums).
//
// The weight's and bias's gradients are sums down the columns.  A thread holds the same
// columns for every row its team takes, so the row pass adds them up in registers, then
// across the teams of the block through shared memory, and leaves one row of partial sums
// per block; norm_grads_kernel adds those up.  The order of every sum is fixed by the
// sizes: no atomics, the same bits every time.
#include <cuda_runtime.h>
#include <stdint.h>

#include "anvil_device.cuh"
#include "anvil_norm.h"
#include "anvil_types.cuh"

namespace anvil {

// Team shapes.  A team of TPR threads holds a row as NV units per thread, where a unit is
// a 16-byte vector (VEC) or one element; unit u of thread t is unit t + u * TPR of the row.
template <typename T, bool VEC, int TPR, int NV>
struct Shape {
    static constexpr int E = VEC ? Elem<T>::VEC : 1;  // elements per unit
    static constexpr int BLOCK = TPR > 256 ? TPR : 256;
    static constexpr int TEAMS = TPR > 32 ? 1 : BLOCK / TPR;
    static constexpr int THREADS = TPR > 32 ? TPR : BLOCK;
    static constexpr int CAP = TPR * NV * E;  // widest row
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* p, float* f) {
    if constexpr (VEC) Elem<T>::unpack(ldg_stream(p), f);
    else f[0] = Elem<T>::load(*p);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* p, const float* f) {
    if constexpr (VEC) stg_stream(p, Elem<T>::pack(f));
    else *p = Elem<T>::store(f[0]);
}
// E weights (fp32 or the rows' type) at column c; cached loads, shared by every row.
template <typename W, int E>
__device__ __forceinline__ void load_weight(const W* w, int c, float* f) {
    if constexpr (E == 1) {
        f[0] = Elem<W>::load(w[c]);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += Elem<W>::VEC) Elem<W>::unpack(__ldg(reinterpret_cast<const uint4*>(w + c + e)), f + e);
    }
}

template <typename T, typename W, bool VEC, int TPR, int NV>
__global__ void __launch_bounds__(Shape<T, VEC, TPR, NV>::THREADS) norm_fwd_kernel(const NormFwdParams p) {
    using S = Shape<T, VEC, TPR, NV>;
    constexpr int E = S::E;
    __shared__ float red[2][TPR > 32 ? TPR / 32 : 1];
    const int t = threadIdx.x % TPR;
    const long long row = blockIdx.x * static_cast<long long>(S::TEAMS) + threadIdx.x / TPR;
    const bool live = row < p.rows;  // a team past the end takes part in the shuffles only
    const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.ldx;
    float v[NV][E];
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (t + u * TPR) * E;
        if (live && c < p.width) {
            load_unit<T, VEC>(x + c, v[u]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) sum += v[u][e];
    const float n = static_cast<float>(p.width);
    const float mean = team_sum<TPR>(sum, red[0]) / n;
    float sq = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if ((t + u * TPR) * E < p.width) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[u][e] -= mean;
                sq += v[u][e] * v[u][e];
            }
        }
    }
    const float rstd = 1.f / sqrtf(team_sum<TPR>(sq, red[1]) / n + p.eps);
    if (!live) return;
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
    const W* w = static_cast<const W*>(p.weight);
    const W* b = static_cast<const W*>(p.bias);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (t + u * TPR) * E;
        if (c >= p.width) break;
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] *= rstd;
        if (w) {
            load_weight<W, E>(w, c, f);
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] *= f[e];
        }
        if (b) {
            load_weight<W, E>(b, c, f);
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] += f[e];
        }
        store_unit<T, VEC>(y + c, v[u]);
    }
}

// A unit as it was loaded, unpacked where it is used: half the registers of fp32 values.
template <typename T, bool VEC>
struct RawUnit {
    uint4 r;
    __device__ __forceinline__ void load(const T* p) { r = ldg_stream(p); }
    __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float* f) const { Elem<T>::unpack(r, f); }
};
template <typename T>
struct RawUnit<T, false> {
    T r;
    __device__ __forceinline__ void load(const T* p) { r = *p; }
    __device__ __forceinline__ void zero() { r = Elem<T>::store(0.f); }
    __device__ __forceinline__ void get(float* f) const { f[0] = Elem<T>::load(r); }
};

// The column sums of a thread: in registers, or (SUMS_SMEM, rows over 8192 wide, whose
// sums would take more registers than the SM has) in shared memory, which no other thread
// of the block touches.
template <typename T, typename W, bool VEC, int TPR, int NV, bool SUMS_SMEM>
__global__ void __launch_bounds__(Shape<T, VEC, TPR, NV>::THREADS) norm_bwd_kernel(const NormBwdParams p) {
    using S = Shape<T, VEC, TPR, NV>;
    constexpr int E = S::E;
    static_assert(!SUMS_SMEM || S::TEAMS == 1, "sums in shared memory are one team's");
    __shared__ float red[2][2][TPR > 32 ? TPR / 32 : 1];
    extern __shared__ __align__(16) float cols[];  // [2][width]
    const int t = threadIdx.x % TPR;
    const int team = threadIdx.x / TPR;
    const float n = static_cast<float>(p.width);
    const W* w = static_cast<const W*>(p.weight);
    constexpr int NA = SUMS_SMEM ? 1 : NV;
    float aw[NA][E], ab[NA][E];
#pragma unroll
    for (int u = 0; u < NA; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) aw[u][e] = ab[u][e] = 0.f;
    if constexpr (SUMS_SMEM) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = (t + u * TPR) * E + e;
                if (c < p.width) cols[c] = cols[p.width + c] = 0.f;
            }
    }
    const long long step = static_cast<long long>(gridDim.x) * S::TEAMS;
    const long long first = blockIdx.x * static_cast<long long>(S::TEAMS);
    using Raw = RawUnit<T, VEC>;
    Raw xr[NV], gr[NV];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](long long row, Raw (&xo)[NV], Raw (&go)[NV], float& mo, float& so) {
        const bool live = row < p.rows;
        const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.ldx;
        const T* dy = static_cast<const T*>(p.dy) + (live ? row : 0) * p.lddy;
        mo = live ? p.mean[row] : 0.f;
        so = live ? p.rstd[row] : 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (t + u * TPR) * E;
            if (live && c < p.width) {
                xo[u].load(x + c);
                go[u].load(dy + c);
            } else {
                xo[u].zero();
                go[u].zero();
            }
        }
    };
    fetch(first + team, xr, gr, mean, rstd);
    int it = 0;
    // every team of the block makes the same number of turns (the reductions are collective)
    for (long long base = first; base < p.rows; base += step, it ^= 1) {
        const long long row = base + team;
        const bool live = row < p.rows;
        // the next row and this row's residual gradient are on their way during the sums
        Raw xn[NV], gn[NV], rr[NV];
        float mean_n = 0.f, rstd_n = 0.f;
        if (base + step < p.rows) fetch(row + step, xn, gn, mean_n, rstd_n);
        if (p.res && live) {
            const T* r = static_cast<const T*>(p.res) + row * p.ldr;
#pragma unroll
            for (int u = 0; u < NV; ++u)
                if ((t + u * TPR) * E < p.width) rr[u].load(r + (t + u * TPR) * E);
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (t + u * TPR) * E;
            if (c >= p.width) break;
            float f[E], h[E], g[E];
            xr[u].get(h);
            gr[u].get(g);
            if (w) {
                load_weight<W, E>(w, c, f);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = 1.f;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[e] = (h[e] - mean) * rstd;
                if constexpr (SUMS_SMEM) {
                    cols[c + e] += g[e] * h[e];
                    cols[p.width + c + e] += g[e];
                } else {
                    aw[u][e] += g[e] * h[e];
                    ab[u][e] += g[e];
                }
                g[e] *= f[e];
                s1 += g[e];
                s2 += g[e] * h[e];
            }
        }
        s1 = team_sum<TPR>(s1, red[it][0]) / n;
        s2 = team_sum<TPR>(s2, red[it][1]) / n;
        if (live && p.dx) {
            T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = (t + u * TPR) * E;
                if (c >= p.width) break;
                float f[E], h[E], g[E];
                xr[u].get(h);
                gr[u].get(g);
                if (w) {
                    load_weight<W, E>(w, c, f);
#pragma unroll
                    for (int e = 0; e < E; ++e) g[e] *= f[e];
                }
                if (p.res) {
                    rr[u].get(f);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) f[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] += rstd * (g[e] - s1 - (h[e] - mean) * rstd * s2);
                store_unit<T, VEC>(dx + c, f);
            }
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            xr[u] = xn[u];
            gr[u] = gn[u];
        }
        mean = mean_n;
        rstd = rstd_n;
    }
    if (!p.dweight && !p.dbias) return;
    // the block's column sums: team 0's registers, then every other team's in turn
    if constexpr (S::TEAMS > 1) {
        for (int k = 1; k < S::TEAMS; ++k) {
            __syncthreads();
            if (team == k) {
#pragma unroll
                for (int u = 0; u < NV; ++u)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int c = (t + u * TPR) * E + e;
                        if (c < p.width) {
                            cols[c] = aw[u][e];
                            cols[p.width + c] = ab[u][e];
                        }
                    }
            }
            __syncthreads();
            if (team == 0) {
#pragma unroll
                for (int u = 0; u < NV; ++u)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int c = (t + u * TPR) * E + e;
                        if (c < p.width) {
                            aw[u][e] += cols[c];
                            ab[u][e] += cols[p.width + c];
                        }
                    }
            }
        }
    }
    if (team != 0) return;
    float* pw = p.blocks > 1 ? p.part + static_cast<size_t>(blockIdx.x) * 2 * p.width : p.dweight;
    float* pb = p.blocks > 1 ? p.part + static_cast<size_t>(blockIdx.x) * 2 * p.width + p.width : p.dbias;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (t + u * TPR) * E + e;
            if (c < p.width) {
                if (p.dweight) pw[c] = SUMS_SMEM ? cols[c] : aw[SUMS_SMEM ? 0 : u][e];
                if (p.dbias) pb[c] = SUMS_SMEM ? cols[p.width + c] : ab[SUMS_SMEM ? 0 : u][e];
            }
        }
}

// dweight (blockIdx.y = 0) and dbias (1): 32 columns per block, 16 threads down each, the
// partial rows taken in order by each and the 16 sums added in order.
constexpr int GRAD_LANES = 16;
__global__ void __launch_bounds__(32 * GRAD_LANES) norm_grads_kernel(const NormBwdParams p) {
    __shared__ float s[GRAD_LANES][32];
    const int x = threadIdx.x & 31, yy = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float* out = blockIdx.y ? p.dbias : p.dweight;
    if (!out) return;
    pdl_wait_previous();
    float a = 0.f;
    if (c < p.width)
        for (int b = yy; b < p.blocks; b += GRAD_LANES)
            a += p.part[(static_cast<size_t>(b) * 2 + blockIdx.y) * p.width + c];
    s[yy][x] = a;
    __syncthreads();
    if (yy == 0 && c < p.width) {
        for (int k = 1; k < GRAD_LANES; ++k) a += s[k][x];
        out[c] = a;
    }
}

namespace {

bool aligned16(const void* p, long long ld, int es, long long rows) {
    return !(reinterpret_cast<uintptr_t>(p) & 15) && (rows <= 1 || (ld * es) % 16 == 0);
}

template <typename T, typename W, bool VEC, int TPR, int NV>
cudaError_t run_fwd(const NormFwdParams& p, cudaStream_t s) {
    using S = Shape<T, VEC, TPR, NV>;
    const long long blocks = (p.rows + S::TEAMS - 1) / S::TEAMS;
    norm_fwd_kernel<T, W, VEC, TPR, NV><<<static_cast<unsigned>(blocks), S::THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename W, bool VEC, int TPR, int NV, bool SUMS_SMEM = false>
cudaError_t run_bwd(const NormBwdParams& p, cudaStream_t s) {
    using S = Shape<T, VEC, TPR, NV>;
    auto kernel = norm_bwd_kernel<T, W, VEC, TPR, NV, SUMS_SMEM>;
    const size_t smem = S::TEAMS > 1 || SUMS_SMEM ? 2 * sizeof(float) * p.width : 0;
    if (SUMS_SMEM) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * sizeof(float) * S::CAP);
        if (e) return e;
    }
    kernel<<<p.blocks, S::THREADS, smem, s>>>(p);
    return cudaGetLastError();
}

// The narrowest team that holds the row: fewer threads per row means fewer barriers and
// more rows in flight per block.  16-byte units where every array is 16-byte aligned row
// by row, single elements otherwise.
template <typename T, typename W>
cudaError_t pick_fwd(const NormFwdParams& p, bool vec, cudaStream_t s) {
    constexpr int E = Elem<T>::VEC;
    const int w = p.width;
    if (vec) {
        if (w <= 8 * E) return run_fwd<T, W, true, 8, 1>(p, s);
        if (w <= 32 * E) return run_fwd<T, W, true, 32, 1>(p, s);
        if (w <= 96 * E) return run_fwd<T, W, true, 32, 3>(p, s);
        if (w <= 256 * E) return run_fwd<T, W, true, 128, 2>(p, s);
        if (w <= 384 * E) return run_fwd<T, W, true, 128, 3>(p, s);
        if (w <= 512 * E) return run_fwd<T, W, true, 128, 4>(p, s);
        if (w <= 1024 * E) return run_fwd<T, W, true, 256, 4>(p, s);
        return run_fwd<T, W, true, 512, 8>(p, s);
    }
    if (w <= 64) return run_fwd<T, W, false, 8, 8>(p, s);
    if (w <= 256) return run_fwd<T, W, false, 32, 8>(p, s);
    if (w <= 1024) return run_fwd<T, W, false, 128, 8>(p, s);
    if (w <= 4096) return run_fwd<T, W, false, 256, 16>(p, s);
    return run_fwd<T, W, false, 512, 32>(p, s);
}

template <typename T, typename W>
cudaError_t pick_bwd(const NormBwdParams& p, bool vec, cudaStream_t s) {
    constexpr int E = Elem<T>::VEC;
    constexpr int NW = 16 / E;  // units of 16 elements per thread
    const int w = p.width;
    if (vec) {
        if (w <= 8 * E) return run_bwd<T, W, true, 8, 1>(p, s);
        if (w <= 32 * E) return run_bwd<T, W, true, 32, 1>(p, s);
        if (w <= 96 * E) return run_bwd<T, W, true, 32, 3>(p, s);
        if (w <= 256 * E) return run_bwd<T, W, true, 128, 2>(p, s);
        if (w <= 384 * E) return run_bwd<T, W, true, 128, 3>(p, s);
        if (w <= 4096) return run_bwd<T, W, true, 256, NW>(p, s);
        if (w <= 8192) return run_bwd<T, W, true, 512, NW>(p, s);
        return run_bwd<T, W, true, 512, 2 * NW, true>(p, s);
    }
    if (w <= 64) return run_bwd<T, W, false, 8, 8>(p, s);
    if (w <= 256) return run_bwd<T, W, false, 32, 8>(p, s);
    if (w <= 1024) return run_bwd<T, W, false, 128, 8>(p, s);
    if (w <= 4096) return run_bwd<T, W, false, 256, 16>(p, s);
    if (w <= 8192) return run_bwd<T, W, false, 512, 16>(p, s);
    return run_bwd<T, W, false, 512, 32, true>(p, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwdParams& p, cudaStream_t s) {
    const int es = dtype_size(p.dtype), ws = dtype_size(p.weight_dtype);
    const int unit = 16 / es;
    const bool vec = p.width % unit == 0 && aligned16(p.x, p.ldx, es, p.rows) && aligned16(p.y, p.ldy, es, p.rows) &&
                     aligned16(p.weight, 0, ws, 1) && aligned16(p.bias, 0, ws, 1);
    switch (p.dtype) {
        case DT_F32: return pick_fwd<float, float>(p, vec, s);
        case DT_BF16:
            return p.weight_dtype == DT_F32 ? pick_fwd<__nv_bfloat16, float>(p, vec, s)
                                            : pick_fwd<__nv_bfloat16, __nv_bfloat16>(p, vec, s);
        default:
            return p.weight_dtype == DT_F32 ? pick_fwd<__half, float>(p, vec, s) : pick_fwd<__half, __half>(p, vec, s);
    }
}

int norm_bwd_blocks(long long rows, int width, int dtype, int sm_count) {
    // narrow rows: teams of 8 or 32 threads, 32 or 8 rows per block and turn; else one row
    const int unit = 16 / dtype_size(dtype);
    const int per_block = width <= 64 ? 32 : width <= 96 * unit ? 8 : 1;
    const long long want = (rows + per_block - 1) / per_block;
    const long long cap = static_cast<long long>(sm_count) * (width <= 256 * unit ? 4 : 2);
    return static_cast<int>(want < 1 ? 1 : want < cap ? want : cap);
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, cudaStream_t s) {
    const int es = dtype_size(p.dtype), ws = dtype_size(p.weight_dtype);
    const int unit = 16 / es;
    const bool vec = p.width % unit == 0 && aligned16(p.x, p.ldx, es, p.rows) && aligned16(p.dy, p.lddy, es, p.rows) &&
                     (!p.dx || aligned16(p.dx, p.lddx, es, p.rows)) && (!p.res || aligned16(p.res, p.ldr, es, p.rows)) &&
                     aligned16(p.weight, 0, ws, 1);
    switch (p.dtype) {
        case DT_F32: return pick_bwd<float, float>(p, vec, s);
        case DT_BF16:
            return p.weight_dtype == DT_F32 ? pick_bwd<__nv_bfloat16, float>(p, vec, s)
                                            : pick_bwd<__nv_bfloat16, __nv_bfloat16>(p, vec, s);
        default:
            return p.weight_dtype == DT_F32 ? pick_bwd<__half, float>(p, vec, s) : pick_bwd<__half, __half>(p, vec, s);
    }
}

cudaError_t launch_norm_grads(const NormBwdParams& p, cudaStream_t s) {
    return launch_pdl(norm_grads_kernel, dim3((p.width + 31) / 32, 2), dim3(32 * GRAD_LANES), 0, s, p);
}

}  // namespace anvil
