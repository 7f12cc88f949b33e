// anvil_norm.cu -- layer norm, forward and backward, for sm_103a.
//
//   forward   mean = sum_j x_j / n,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / n + eps),
//             y_j = (x_j - mean) rstd w_j + b_j
//   backward  h_j = (x_j - mean) rstd,  g_j = dy_j w_j,
//             dx_j = rstd (g_j - mean_j(g) - h_j mean_j(g h)) [+ r_j],
//             dw_j = sum over rows of dy_j h_j,  db_j = sum over rows of dy_j
//
// Both passes read each input once and write each output once, so HBM bounds them.  A row
// belongs to a team of threads that keeps it in registers, as it was loaded, between the
// reductions and the store (the variance is taken from the centred values, in a second pass
// over registers, not from a difference of large sums).  A block takes row after row, so a
// thread has the same columns every time: it holds their weights in registers (loaded again
// for every row, fp32 weights of 16-bit rows were four of the six 16-byte accesses per
// vector, and shared memory's pipe the bound), and the next row's loads go out before this
// row's sums.
//
// The weight's and bias's gradients are sums down the columns: a thread adds up its columns
// in registers, the teams of a block join theirs through shared memory, and each block
// leaves one row of partial sums; norm_grads_kernel adds those up.  The order of every sum
// is fixed by the sizes: no atomics, the same bits every time.
//
// Many rows (the ring kernels): the rows come by bulk copies into a ring of shared-memory
// stages per team, several rows ahead.  With one row ahead in registers a block waited out
// the memory's latency on every row (32768 x 2816 bf16: 150-168 us backward, 78 forward;
// with the ring 121-125 and 65, 5.7-6.1 TB/s; 32768 x 2815, off the 16-byte boundaries,
// backward: 522, with the ring 199; forward, without it, 152: bound by the instructions of
// element-by-element accesses, 2.4 TB/s; results staged in shared memory and stored by bulk
// copies were slower, 227 backward).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "anvil_device.cuh"
#include "anvil_host.h"
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

// Resident blocks per SM: the backward row pass 512 threads, at up to 128 registers each;
// the forward one 1024 threads at 64 where a thread has at most 8 columns, 768 at 85 up to 16,
// else 512 (teams of up to a warp: three blocks of 256).
constexpr int bwd_blocks_per_sm(int tpr) { return tpr <= 32 ? 2 : 512 / tpr; }
constexpr int fwd_threads_per_sm(int columns) { return columns <= 8 ? 1024 : columns <= 16 ? 768 : 512; }
constexpr int fwd_blocks_per_sm(int tpr, int columns) {
    return tpr <= 32 ? 3 : tpr < fwd_threads_per_sm(columns) ? fwd_threads_per_sm(columns) / tpr : 1;
}

// A unit as it was loaded, unpacked where it is used (half the registers of fp32 values of
// 16-bit types), and the arithmetic on it: packed fp32 pairs for vectors, one value else.
template <typename T, bool VEC>
struct RawUnit {
    static constexpr int P = Elem<T>::VEC / 2;
    using F = uint64_t;
    uint4 r;
    __device__ __forceinline__ void load(const T* p) { r = ldg_stream(p); }
    __device__ __forceinline__ void load_shared(uint32_t a) { r = lds128(a); }
    __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(F* f) const { Elem<T>::unpack_pairs(r, f); }
    static __device__ __forceinline__ void put(T* p, const F* f) { stg_stream(p, Elem<T>::pack_pairs(f)); }
};
template <typename T>
struct RawUnit<T, false> {
    static constexpr int P = 1;
    using F = float;
    T r;
    __device__ __forceinline__ void load(const T* p) { r = __ldcs(p); }
    __device__ __forceinline__ void load_shared(uint32_t a) {
        if constexpr (sizeof(T) == 2) {
            uint16_t b;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(a) : "memory");
            memcpy(&r, &b, 2);
        } else {
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
        }
    }
    __device__ __forceinline__ void zero() { r = Elem<T>::store(0.f); }
    __device__ __forceinline__ void get(F* f) const { f[0] = Elem<T>::load(r); }
    static __device__ __forceinline__ void put(T* p, const F* f) { __stcs(p, Elem<T>::store(f[0])); }
};
__device__ __forceinline__ float p_add(float a, float b) { return a + b; }
__device__ __forceinline__ float p_mul(float a, float b) { return a * b; }
__device__ __forceinline__ float p_fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float p_sum(float a) { return a; }
__device__ __forceinline__ uint64_t p_add(uint64_t a, uint64_t b) { return f2_add(a, b); }
__device__ __forceinline__ uint64_t p_mul(uint64_t a, uint64_t b) { return f2_mul(a, b); }
__device__ __forceinline__ uint64_t p_fma(uint64_t a, uint64_t b, uint64_t c) { return f2_fma(a, b, c); }
__device__ __forceinline__ float p_sum(uint64_t a) {
    float lo, hi;
    f2_split(a, &lo, &hi);
    return lo + hi;
}
// 1 / sqrt(v): the hardware's estimate (2 ulp) and one Newton step.
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = rsqrtf(v);
    return v > 0.f && v < INFINITY ? fmaf(0.5f * r, fmaf(-v * r, r, 1.f), r) : r;
}
template <typename F>
__device__ __forceinline__ F p_all(float v) {
    if constexpr (sizeof(F) == 8) return f2_make(v, v);
    else return v;
}
template <typename F>
__device__ __forceinline__ void p_split(F v, float* f) {
    if constexpr (sizeof(F) == 8) f2_split(v, f, f + 1);
    else f[0] = v;
}

// E weights (fp32 or the rows' type) at column c.
template <typename W, int E>
__device__ __forceinline__ void load_weight(const W* w, int c, float* f) {
    if constexpr (E == 1) {
        f[0] = Elem<W>::load(w[c]);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += Elem<W>::VEC) Elem<W>::unpack(*reinterpret_cast<const uint4*>(w + c + e), f + e);
    }
}
// A unit's columns of an optional weight vector (null: every value is `none`).
template <typename W, int E, typename F>
__device__ __forceinline__ void weight_unit(const W* w, int c, int width, float none, F* f) {
    if (w && c < width) {
        float v[E];
        load_weight<W, E>(w, c, v);
        if constexpr (sizeof(F) == 8) {
#pragma unroll
            for (int e = 0; e < E; e += 2) f[e / 2] = f2_make(v[e], v[e + 1]);
        } else {
            f[0] = v[0];
        }
    } else {
#pragma unroll
        for (int e = 0; e < (sizeof(F) == 8 ? E / 2 : 1); ++e) f[e] = p_all<F>(none);
    }
}

template <typename T, typename W, bool VEC, int TPR, int NV>
__global__ void __launch_bounds__(Shape<T, VEC, TPR, NV>::THREADS, fwd_blocks_per_sm(TPR, NV * Shape<T, VEC, TPR, NV>::E))
    norm_fwd_kernel(const NormFwdParams p) {
    using S = Shape<T, VEC, TPR, NV>;
    using Raw = RawUnit<T, VEC>;
    constexpr int E = S::E;
    __shared__ __align__(16) float red[2][2][TPR > 32 ? TPR / 32 : 4];
    const int t = threadIdx.x % TPR;
    const int team = threadIdx.x / TPR;
    const float inv_n = 1.f / static_cast<float>(p.width);
    constexpr int P = Raw::P;
    using F = typename Raw::F;
    pdl_allow_next();
    pdl_wait_previous();
    F w[NV][P], b[NV][P];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        weight_unit<W, E>(static_cast<const W*>(p.weight), (t + u * TPR) * E, p.width, 1.f, w[u]);
        weight_unit<W, E>(static_cast<const W*>(p.bias), (t + u * TPR) * E, p.width, 0.f, b[u]);
    }
    bool in[NV];  // which of this thread's units lie in the row
#pragma unroll
    for (int u = 0; u < NV; ++u) in[u] = (t + u * TPR) * E < p.width;
    const long long step = static_cast<long long>(gridDim.x) * S::TEAMS;
    const long long first = blockIdx.x * static_cast<long long>(S::TEAMS);
    long long row = first + team;
    // this thread's first unit of the row to be loaded next, and of the row to be stored
    const T* xp = static_cast<const T*>(p.x) + row * p.ldx + t * E;
    T* yp = static_cast<T*>(p.y) + row * p.ldy + t * E;
    const long long xstep = step * p.ldx, ystep = step * p.ldy;
    auto fetch = [&](bool live, Raw (&xo)[NV]) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (live && in[u]) xo[u].load(xp + u * TPR * E);
            else xo[u].zero();
        }
        xp += xstep;
    };
    Raw xr[NV], xn[NV];
    fetch(row < p.rows, xr);
    int it = 0;
    // every team of the block makes the same number of turns (the reductions are collective)
    for (long long base = first; base < p.rows; base += step, row += step, yp += ystep, it ^= 1) {
        fetch(row + step < p.rows, xn);
        F acc = p_all<F>(0.f);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            F v[P];
            xr[u].get(v);
#pragma unroll
            for (int i = 0; i < P; ++i) acc = p_add(acc, v[i]);
        }
        const float mean = team_sum<TPR>(p_sum(acc), red[it][0]) * inv_n;
        const F nm = p_all<F>(-mean);
        acc = p_all<F>(0.f);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (in[u]) {
                F v[P];
                xr[u].get(v);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F d = p_add(v[i], nm);
                    acc = p_fma(d, d, acc);
                }
            }
        }
        const float rstd = inv_sqrt(fmaf(team_sum<TPR>(p_sum(acc), red[it][1]), inv_n, p.eps));
        if (row < p.rows) {
            if (t == 0) {
                if (p.mean) p.mean[row] = mean;
                if (p.rstd) p.rstd[row] = rstd;
            }
            const F rs = p_all<F>(rstd);
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                if (!in[u]) break;
                F v[P];
                xr[u].get(v);
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = p_fma(p_mul(p_add(v[i], nm), rs), w[u][i], b[u][i]);
                Raw::put(yp + u * TPR * E, v);
            }
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) xr[u] = xn[u];
    }
}

// The column sums of a thread: in registers, or (SUMS_SMEM, rows over 8192 wide, whose
// sums would take more registers than the SM has) in shared memory, which no other thread
// of the block touches; such a block reads its weights for every row.  4096 x 16384 bf16: 146
// us (sums laid out by column, a lane's eight neighbours: 319, the banks' conflicts).
template <typename T, typename W, bool VEC, int TPR, int NV, bool SUMS_SMEM>
__global__ void __launch_bounds__(Shape<T, VEC, TPR, NV>::THREADS, bwd_blocks_per_sm(TPR))
    norm_bwd_kernel(const NormBwdParams p) {
    using S = Shape<T, VEC, TPR, NV>;
    using Raw = RawUnit<T, VEC>;
    constexpr int E = S::E;
    static_assert(!SUMS_SMEM || S::TEAMS == 1, "sums in shared memory are one team's");
    __shared__ __align__(16) float2 red[2][TPR > 32 ? TPR / 32 : 2];
    extern __shared__ __align__(16) float cols[];  // [2][width]
    const int t = threadIdx.x % TPR;
    const int team = threadIdx.x / TPR;
    const float inv_n = 1.f / static_cast<float>(p.width);
    const W* w = static_cast<const W*>(p.weight);
    constexpr int P = Raw::P;
    using F = typename Raw::F;
    constexpr int NA = SUMS_SMEM ? 1 : NV;
    F aw[NA][P], ab[NA][P], wv[NA][P];
    pdl_allow_next();
    pdl_wait_previous();
    // SUMS_SMEM: the thread's sums of unit u, pair i at own[(u * P + i) * TPR]: neighbouring lanes
    // at neighbouring addresses
    struct alignas(2 * sizeof(F)) Sums {
        F w, b;
    };
    Sums* own = reinterpret_cast<Sums*>(cols) + t;
    if constexpr (SUMS_SMEM) {
#pragma unroll
        for (int i = 0; i < NV * P; ++i) own[i * TPR] = {p_all<F>(0.f), p_all<F>(0.f)};
    } else {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            weight_unit<W, E>(w, (t + u * TPR) * E, p.width, 1.f, wv[u]);
#pragma unroll
            for (int i = 0; i < P; ++i) aw[u][i] = ab[u][i] = p_all<F>(0.f);
        }
    }
    auto weight_of = [&](int u, F (&f)[P]) {
        if constexpr (SUMS_SMEM) {
            weight_unit<W, E>(w, (t + u * TPR) * E, p.width, 1.f, f);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = wv[u][i];
        }
    };
    bool in[NV];  // which of this thread's units lie in the row
#pragma unroll
    for (int u = 0; u < NV; ++u) in[u] = (t + u * TPR) * E < p.width;
    const long long step = static_cast<long long>(gridDim.x) * S::TEAMS;
    const long long first = blockIdx.x * static_cast<long long>(S::TEAMS);
    long long row = first + team;
    // this thread's first unit: of the row to be loaded next (x, dy), of this row (res, dx)
    const T* xp = static_cast<const T*>(p.x) + row * p.ldx + t * E;
    const T* gp = static_cast<const T*>(p.dy) + row * p.lddy + t * E;
    const T* rp = static_cast<const T*>(p.res) + row * p.ldr + t * E;
    T* dp = static_cast<T*>(p.dx) + row * p.lddx + t * E;
    const long long xstep = step * p.ldx, gstep = step * p.lddy, rstep = step * p.ldr, dstep = step * p.lddx;
    Raw xr[NV], gr[NV];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](long long r, Raw (&xo)[NV], Raw (&go)[NV], float& mo, float& so) {
        const bool live = r < p.rows;
        mo = live ? p.mean[r] : 0.f;
        so = live ? p.rstd[r] : 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (live && in[u]) {
                xo[u].load(xp + u * TPR * E);
                go[u].load(gp + u * TPR * E);
            } else {
                xo[u].zero();
                go[u].zero();
            }
        }
        xp += xstep;
        gp += gstep;
    };
    fetch(row, xr, gr, mean, rstd);
    int it = 0;
    // every team of the block makes the same number of turns (the reductions are collective)
    for (long long base = first; base < p.rows; base += step, row += step, rp += rstep, dp += dstep, it ^= 1) {
        const bool live = row < p.rows;
        Raw xn[NV], gn[NV], rr[NV];
        float mean_n = 0.f, rstd_n = 0.f;
        fetch(row + step, xn, gn, mean_n, rstd_n);
        if (p.res && live) {
#pragma unroll
            for (int u = 0; u < NV; ++u)
                if (in[u]) rr[u].load(rp + u * TPR * E);
        }
        const F nm = p_all<F>(-mean), rs = p_all<F>(rstd);
        F a1 = p_all<F>(0.f), a2 = p_all<F>(0.f);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (!in[u]) break;
            F f[P], h[P], g[P];
            xr[u].get(h);
            gr[u].get(g);
            weight_of(u, f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                h[i] = p_mul(p_add(h[i], nm), rs);
                if constexpr (SUMS_SMEM) {
                    Sums q = own[(u * P + i) * TPR];
                    q.w = p_fma(g[i], h[i], q.w);
                    q.b = p_add(q.b, g[i]);
                    own[(u * P + i) * TPR] = q;
                } else {
                    aw[u][i] = p_fma(g[i], h[i], aw[u][i]);
                    ab[u][i] = p_add(ab[u][i], g[i]);
                }
                g[i] = p_mul(g[i], f[i]);
                a1 = p_add(a1, g[i]);
                a2 = p_fma(g[i], h[i], a2);
            }
        }
        float s1 = p_sum(a1), s2 = p_sum(a2);
        team_sum2<TPR>(s1, s2, red[it]);
        if (live && p.dx) {
            // rstd (g - s1 - h s2) = rstd g - (rstd s1) - h (rstd s2)
            const F k1 = p_all<F>(-rstd * (s1 * inv_n)), k2 = p_all<F>(-rstd * (s2 * inv_n));
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                if (!in[u]) break;
                F f[P], h[P], g[P];
                xr[u].get(h);
                gr[u].get(g);
                weight_of(u, f);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    h[i] = p_fma(p_mul(p_add(h[i], nm), rs), k2, k1);
                    g[i] = p_fma(p_mul(g[i], f[i]), rs, h[i]);
                }
                if (p.res) {
                    rr[u].get(f);
#pragma unroll
                    for (int i = 0; i < P; ++i) g[i] = p_add(g[i], f[i]);
                }
                Raw::put(dp + u * TPR * E, g);
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
    float cw[NV][E], cb[NV][E];
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < P; ++i) {
            p_split(SUMS_SMEM ? own[(u * P + i) * TPR].w : aw[SUMS_SMEM ? 0 : u][i], &cw[u][i * (E / P)]);
            p_split(SUMS_SMEM ? own[(u * P + i) * TPR].b : ab[SUMS_SMEM ? 0 : u][i], &cb[u][i * (E / P)]);
        }
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
                            cols[c] = cw[u][e];
                            cols[p.width + c] = cb[u][e];
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
                            cw[u][e] += cols[c];
                            cb[u][e] += cols[p.width + c];
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
                if (p.dweight) pw[c] = cw[u][e];
                if (p.dbias) pb[c] = cb[u][e];
            }
        }
}

// ---------------------------------------------------------------- the ring kernels
// A team of TPR threads (64 to 512) takes a run of consecutive rows; up to RING_MAX stages
// of `arrays` rows each (x, or x, dy and the residual's gradient) are on their way.  The
// team's first thread issues the copies of a stage once the team has read what was in it.
//
// Rows off the 16-byte boundaries (VEC false, backward only; forward the plain kernels are as
// fast): a bulk copy takes the 16-byte pieces that cover the row, so it brings up to 14
// bytes of the rows (or padding) before and after, which nothing reads; the array's first and
// last row, which have no such neighbour on one side, are copied element by element.  A
// thread then has every TPR-th element.
constexpr int RING_MAX = 8;
constexpr int RING_BLOCK = 256;                  // threads per block, about (512 where a team is that wide)
constexpr int RING_BYTES = 200 * 1024;           // shared memory of an SM's blocks
// Blocks per SM: two of 256 threads, three of 192 (32768 x 2816 bf16 forward: 65 us, 70 with
// two; three of 256 threads were slower, 48 against 45 at 65536 x 1024).
constexpr int ring_blocks(int tpr) { return tpr > RING_BLOCK ? 1 : tpr == 192 ? 3 : 2; }
constexpr int ring_teams(int tpr) { return tpr > RING_BLOCK ? 1 : RING_BLOCK / tpr; }
constexpr int ring_threads(int tpr) { return ring_teams(tpr) * tpr; }
constexpr int ring_bytes(int tpr) { return RING_BYTES / ring_blocks(tpr) / 1024 * 1024; }
// Bytes of a row's place in a stage.
__host__ __device__ constexpr int ring_slot(bool vec, int row_bytes) { return vec ? row_bytes : (row_bytes + 31) / 16 * 16; }
// Stages per team of a ring of `arrays` rows of `row_bytes` (their slots) each.
__host__ __device__ constexpr int ring_stages(int tpr, int arrays, int row_bytes) {
    const int s = (ring_bytes(tpr) - 1024) / ring_teams(tpr) / (arrays * row_bytes);
    return s > RING_MAX ? RING_MAX : s;
}

template <int TPR>
struct Team {
    int id, t;  // of the block's teams; thread of the team
    float4* red;  // [2][TPR / 64] pairs of two warps' sums
    int flip;
    __device__ __forceinline__ void sync() const {
        named_barrier_sync(1 + id, TPR);
    }
    // Sums of a and b over the team, the same in every thread; a barrier of the team.
    __device__ __forceinline__ void sum(float& a, float& b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        // two arrays in turn: one is written again only after the next sum's barrier
        float4* r = red + flip * (TPR / 64);
        flip ^= 1;
        if ((t & 31) == 0) reinterpret_cast<float2*>(r)[t >> 5] = make_float2(a, b);
        sync();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) {
            const float4 f = r[w];
            a += f.x;
            b += f.y;
            a += f.z;
            b += f.w;
        }
    }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// One row (of `rows`) into its slot at `dst` (16-byte aligned): the bytes of bulk copies to
// expect, and the copies.  A row of whole 16-byte pieces starts at the slot's start, others
// at their own offset to a 16-byte boundary.
__device__ __forceinline__ uint32_t slot_offset(const void* row) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15);
}
__device__ __forceinline__ uint32_t cover_bytes(const void* row, uint32_t bytes) {
    return (slot_offset(row) + bytes + 15u) & ~15u;
}
__device__ __forceinline__ void cover_load(uint32_t dst, const void* row, uint32_t bytes, uint64_t* bar) {
    bulk_load(dst, reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(row) & ~static_cast<uintptr_t>(15)),
              cover_bytes(row, bytes), bar);
}
// The same by the team's threads (the array's first and last row).
template <typename T, int TPR>
__device__ __forceinline__ void copy_row(uint32_t dst, const T* row, int width, int t) {
    dst += slot_offset(row);
    for (int i = t; i < width; i += TPR) {
        if constexpr (sizeof(T) == 2) {
            uint16_t b;
            memcpy(&b, row + i, 2);
            sts16(dst + 2 * i, b);
        } else {
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + 4 * i), "f"(row[i]) : "memory");
        }
    }
}

// After a wait that gave up: the copies of `rows` rows into `stages` stages, waited for once
// more before the block's shared memory goes away.
__device__ __forceinline__ void drain(uint64_t* full, int stages, long long rows, unsigned* err) {
    for (int s = 0; s < stages && s < rows; ++s) mbar_wait(&full[s], static_cast<uint32_t>((rows - 1 - s) / stages) & 1u, err);
}

// One row's statistics per lane, 32 rows at a time, the next 32 on their way.
struct RowStats {
    float mean, rstd, mean_n, rstd_n;
    __device__ __forceinline__ void start(const NormBwdParams& p, long long row, long long end, int lane) {
        mean = row + lane < end ? p.mean[row + lane] : 0.f;
        rstd = row + lane < end ? p.rstd[row + lane] : 0.f;
        next(p, row + 32, end, lane);
    }
    __device__ __forceinline__ void next(const NormBwdParams& p, long long row, long long end, int lane) {
        mean_n = row + lane < end ? p.mean[row + lane] : 0.f;
        rstd_n = row + lane < end ? p.rstd[row + lane] : 0.f;
    }
};

template <typename T, typename W, bool VEC, int TPR, int NV>
__global__ void __launch_bounds__(ring_threads(TPR), ring_blocks(TPR)) norm_bwd_ring_kernel(const NormBwdParams p) {
    using Raw = RawUnit<T, VEC>;
    using F = typename Raw::F;
    constexpr int E = VEC ? Elem<T>::VEC : 1, P = Raw::P, TEAMS = ring_teams(TPR);
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t full[TEAMS][RING_MAX];
    __shared__ float4 red[TEAMS][2][TPR / 64];
    const int lane = threadIdx.x & 31;
    Team<TPR> team;
    team.id = threadIdx.x / TPR;
    team.t = threadIdx.x % TPR;
    team.red = &red[team.id][0][0];
    team.flip = 0;
    const int row_bytes = p.width * static_cast<int>(sizeof(T));
    const int arrays = p.res ? 3 : 2;
    const int slot = ring_slot(VEC, row_bytes);
    const int stages = ring_stages(TPR, arrays, slot);
    const uint32_t stage_bytes = static_cast<uint32_t>(arrays * slot);
    uint8_t* mine = ring + static_cast<size_t>(team.id) * stages * stage_bytes;
    const long long g = static_cast<long long>(blockIdx.x) * TEAMS + team.id;
    const long long r0 = g * p.team_rows < p.rows ? g * p.team_rows : p.rows;
    const long long r1 = r0 + p.team_rows < p.rows ? r0 + p.team_rows : p.rows;
    if (threadIdx.x == 0) {
        for (int k = 0; k < TEAMS; ++k)
            for (int s = 0; s < RING_MAX; ++s) mbar_init(&full[k][s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto issue = [&](long long row, int s) {
        uint64_t* bar = &full[team.id][s];
        const uint32_t dst = smem_u32(mine + s * stage_bytes);
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
        const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
        const T* res = static_cast<const T*>(p.res) + row * p.ldr;
        if constexpr (VEC) {
            mbar_arrive_expect_tx(bar, stage_bytes);
            bulk_load(dst, x, row_bytes, bar);
            bulk_load(dst + slot, dy, row_bytes, bar);
            if (p.res) bulk_load(dst + 2 * slot, res, row_bytes, bar);
        } else if (row == 0 || row == p.rows - 1) {
            mbar_arrive_cta(bar);  // the team copies this row when it comes to it
        } else {
            mbar_arrive_expect_tx(bar, cover_bytes(x, row_bytes) + cover_bytes(dy, row_bytes) +
                                           (p.res ? cover_bytes(res, row_bytes) : 0u));
            cover_load(dst, x, row_bytes, bar);
            cover_load(dst + slot, dy, row_bytes, bar);
            if (p.res) cover_load(dst + 2 * slot, res, row_bytes, bar);
        }
    };
    pdl_allow_next();
    pdl_wait_previous();
    if (team.t == 0)
        for (int s = 0; s < stages && r0 + s < r1; ++s) issue(r0 + s, s);
    RowStats st;
    st.start(p, r0, r1, lane);
    const float inv_n = 1.f / static_cast<float>(p.width);
    bool in[NV];
    F aw[NV][P], ab[NV][P], wv[NV][P];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (team.t + u * TPR) * E;
        in[u] = c < p.width;
        weight_unit<W, E>(static_cast<const W*>(p.weight), c, p.width, 1.f, wv[u]);
#pragma unroll
        for (int i = 0; i < P; ++i) aw[u][i] = ab[u][i] = p_all<F>(0.f);
    }
    T* dp = static_cast<T*>(p.dx) + r0 * p.lddx + team.t * E;
    bool dead = false;  // a wait gave up: the rest runs to its end without waiting
    int s = 0;
    uint32_t phase = 0;
    for (long long row = r0; row < r1; ++row, dp += p.lddx) {
        const int k = static_cast<int>(row - r0) & 31;
        if (k == 0 && row != r0) {
            st.mean = st.mean_n;
            st.rstd = st.rstd_n;
            st.next(p, row + 32, r1, lane);
        }
        const float mean = __shfl_sync(0xffffffffu, st.mean, k), rstd = __shfl_sync(0xffffffffu, st.rstd, k);
        if (!dead) dead = !mbar_wait(&full[team.id][s], phase, p.err);
        const uint32_t src = smem_u32(mine + s * stage_bytes);
        uint32_t ox = 0, og = 0, orr = 0;  // the rows' offsets in their slots
        if constexpr (!VEC) {
            const T* x = static_cast<const T*>(p.x) + row * p.ldx;
            const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
            const T* res = static_cast<const T*>(p.res) + row * p.ldr;
            ox = slot_offset(x);
            og = slot_offset(dy);
            orr = slot_offset(res);
            if (row == 0 || row == p.rows - 1) {
                copy_row<T, TPR>(src, x, p.width, team.t);
                copy_row<T, TPR>(src + slot, dy, p.width, team.t);
                if (p.res) copy_row<T, TPR>(src + 2 * slot, res, p.width, team.t);
                fence_proxy_async_smem();  // before the next bulk copies into the stage
                team.sync();
            }
        }
        constexpr uint32_t UNIT = E * sizeof(T);
        Raw xr[NV], gr[NV], rr[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (!in[u]) break;
            const uint32_t at = src + (team.t + u * TPR) * UNIT;
            xr[u].load_shared(at + ox);
            gr[u].load_shared(at + slot + og);
            if (p.res) rr[u].load_shared(at + 2 * slot + orr);
        }
        const F nm = p_all<F>(-mean), rs = p_all<F>(rstd);
        F a1 = p_all<F>(0.f), a2 = p_all<F>(0.f);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (!in[u]) break;
            F h[P], d[P];
            xr[u].get(h);
            gr[u].get(d);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                h[i] = p_mul(p_add(h[i], nm), rs);
                aw[u][i] = p_fma(d[i], h[i], aw[u][i]);
                ab[u][i] = p_add(ab[u][i], d[i]);
                d[i] = p_mul(d[i], wv[u][i]);
                a1 = p_add(a1, d[i]);
                a2 = p_fma(d[i], h[i], a2);
            }
        }
        float s1 = p_sum(a1), s2 = p_sum(a2);
        team.sum(s1, s2);
        // every thread of the team has read the stage
        if (team.t == 0 && row + stages < r1) issue(row + stages, s);
        if (++s == stages) {
            s = 0;
            phase ^= 1u;
        }
        if (!p.dx) continue;
        // rstd (g - s1 - h s2) = rstd g - (rstd s1) - h (rstd s2)
        const F k1 = p_all<F>(-rstd * (s1 * inv_n)), k2 = p_all<F>(-rstd * (s2 * inv_n));
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (!in[u]) break;
            F h[P], d[P];
            xr[u].get(h);
            gr[u].get(d);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                h[i] = p_fma(p_mul(p_add(h[i], nm), rs), k2, k1);
                d[i] = p_fma(p_mul(d[i], wv[u][i]), rs, h[i]);
            }
            if (p.res) {
                rr[u].get(h);
#pragma unroll
                for (int i = 0; i < P; ++i) d[i] = p_add(d[i], h[i]);
            }
            Raw::put(dp + u * TPR * E, d);
        }
    }
    if (dead) drain(full[team.id], stages, r1 - r0, p.err);
    if (!p.dweight && !p.dbias) return;
    // the block's column sums, team by team in order, in the ring (every copy has been read)
    float* cols = reinterpret_cast<float*>(ring);
    for (int k = 0; k < TEAMS; ++k) {
        __syncthreads();
        if (team.id != k) continue;
        const bool last = k == TEAMS - 1;
        float* pw = p.blocks > 1 ? p.part + static_cast<size_t>(blockIdx.x) * 2 * p.width : p.dweight;
        float* pb = p.blocks > 1 ? p.part + static_cast<size_t>(blockIdx.x) * 2 * p.width + p.width : p.dbias;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (!in[u]) break;
            const int c = (team.t + u * TPR) * E;
            float w[E], b[E];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                p_split(aw[u][i], &w[(E / P) * i]);
                p_split(ab[u][i], &b[(E / P) * i]);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (k > 0) {
                    w[e] += cols[c + e];
                    b[e] += cols[p.width + c + e];
                }
                if (!last) {
                    cols[c + e] = w[e];
                    cols[p.width + c + e] = b[e];
                } else {
                    if (p.dweight) pw[c + e] = w[e];
                    if (p.dbias) pb[c + e] = b[e];
                }
            }
        }
    }
}

template <typename T, typename W, int TPR, int NV>
__global__ void __launch_bounds__(ring_threads(TPR), ring_blocks(TPR)) norm_fwd_ring_kernel(const NormFwdParams p) {
    using Raw = RawUnit<T, true>;
    constexpr int E = Elem<T>::VEC, P = E / 2, TEAMS = ring_teams(TPR);
    using F = uint64_t;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t full[TEAMS][RING_MAX];
    __shared__ float4 red[TEAMS][2][TPR / 64];
    Team<TPR> team;
    team.id = threadIdx.x / TPR;
    team.t = threadIdx.x % TPR;
    team.red = &red[team.id][0][0];
    team.flip = 0;
    const uint32_t row_bytes = static_cast<uint32_t>(p.width * sizeof(T));
    const int stages = ring_stages(TPR, 1, row_bytes);
    uint8_t* mine = ring + static_cast<size_t>(team.id) * stages * row_bytes;
    const long long g = static_cast<long long>(blockIdx.x) * TEAMS + team.id;
    const long long r0 = g * p.team_rows < p.rows ? g * p.team_rows : p.rows;
    const long long r1 = r0 + p.team_rows < p.rows ? r0 + p.team_rows : p.rows;
    if (threadIdx.x == 0) {
        for (int k = 0; k < TEAMS; ++k)
            for (int s = 0; s < RING_MAX; ++s) mbar_init(&full[k][s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto issue = [&](long long row, int s) {
        uint64_t* bar = &full[team.id][s];
        mbar_arrive_expect_tx(bar, row_bytes);
        bulk_load(smem_u32(mine + s * row_bytes), static_cast<const T*>(p.x) + row * p.ldx, row_bytes, bar);
    };
    pdl_allow_next();
    pdl_wait_previous();
    if (team.t == 0)
        for (int s = 0; s < stages && r0 + s < r1; ++s) issue(r0 + s, s);
    const float inv_n = 1.f / static_cast<float>(p.width);
    bool in[NV];
    F w[NV][P], b[NV][P];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (team.t + u * TPR) * E;
        in[u] = c < p.width;
        weight_unit<W, E>(static_cast<const W*>(p.weight), c, p.width, 1.f, w[u]);
        weight_unit<W, E>(static_cast<const W*>(p.bias), c, p.width, 0.f, b[u]);
    }
    T* yp = static_cast<T*>(p.y) + r0 * p.ldy + team.t * E;
    bool dead = false;  // a wait gave up: the rest runs to its end without waiting
    int s = 0;
    uint32_t phase = 0;
    // two rows at a time: their sums share the team's barriers
    for (long long row = r0; row < r1; row += 2, yp += 2 * p.ldy) {
        const bool two = row + 1 < r1;
        Raw xr[2][NV];
        int freed[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            freed[k] = s;
            if (k == 0 || two) {
                if (!dead) dead = !mbar_wait(&full[team.id][s], phase, p.err);
                const uint32_t src = smem_u32(mine + s * row_bytes) + team.t * 16;
#pragma unroll
                for (int u = 0; u < NV; ++u) {
                    if (!in[u]) break;
                    xr[k][u].r = lds128(src + u * TPR * 16);
                }
                if (++s == stages) {
                    s = 0;
                    phase ^= 1u;
                }
            } else {
#pragma unroll
                for (int u = 0; u < NV; ++u) xr[k][u].zero();
            }
        }
        float sum[2], sq[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            F acc = 0;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                if (!in[u]) break;
                F v[P];
                xr[k][u].get(v);
#pragma unroll
                for (int i = 0; i < P; ++i) acc = p_add(acc, v[i]);
            }
            sum[k] = p_sum(acc);
        }
        team.sum(sum[0], sum[1]);
        // every thread of the team has read the stages
        if (team.t == 0) {
            if (row + stages < r1) issue(row + stages, freed[0]);
            if (row + 1 + stages < r1) issue(row + 1 + stages, freed[1]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            sum[k] *= inv_n;
            const F nm = p_all<F>(-sum[k]);
            F acc = 0;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                if (!in[u]) break;
                F v[P];
                xr[k][u].get(v);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F d = p_add(v[i], nm);
                    acc = p_fma(d, d, acc);
                }
            }
            sq[k] = p_sum(acc);
        }
        team.sum(sq[0], sq[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 1 && !two) break;
            const float rstd = inv_sqrt(fmaf(sq[k], inv_n, p.eps));
            if (team.t == 0) {
                if (p.mean) p.mean[row + k] = sum[k];
                if (p.rstd) p.rstd[row + k] = rstd;
            }
            const F nm = p_all<F>(-sum[k]), rs = p_all<F>(rstd);
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                if (!in[u]) break;
                F v[P];
                xr[k][u].get(v);
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = p_fma(p_mul(p_add(v[i], nm), rs), w[u][i], b[u][i]);
                Raw::put(yp + k * p.ldy + u * TPR * E, v);
            }
        }
    }
    if (dead) drain(full[team.id], stages, r1 - r0, p.err);
}

// dweight (blockIdx.y = 0) and dbias (1): 32 columns per block, 16 threads down each, the
// partial rows taken in order by each and the 16 sums added in order.
constexpr int GRAD_LANES = 16;
__global__ void __launch_bounds__(32 * GRAD_LANES) norm_grads_kernel(const NormBwdParams p) {
    __shared__ float s[GRAD_LANES][32];
    const int x = threadIdx.x & 31, yy = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float* out = blockIdx.y ? p.dbias : p.dweight;
    pdl_allow_next();
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

template <typename T, typename W, bool VEC, int TPR, int NV>
cudaError_t run_fwd(const NormFwdParams& p, cudaStream_t s) {
    using S = Shape<T, VEC, TPR, NV>;
    const long long want = (p.rows + S::TEAMS - 1) / S::TEAMS;
    const long long cap = 152ll * fwd_blocks_per_sm(TPR, NV * S::E);  // one wave of resident blocks
    const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
    return launch_pdl(norm_fwd_kernel<T, W, VEC, TPR, NV>, grid, dim3(S::THREADS), 0, s, p);
}

template <typename T, typename W, bool VEC, int TPR, int NV, bool SUMS_SMEM = false>
cudaError_t run_bwd(const NormBwdParams& p, cudaStream_t s) {
    using S = Shape<T, VEC, TPR, NV>;
    auto kernel = norm_bwd_kernel<T, W, VEC, TPR, NV, SUMS_SMEM>;
    const size_t smem = SUMS_SMEM ? 2 * sizeof(float) * S::CAP : S::TEAMS > 1 ? 2 * sizeof(float) * p.width : 0;
    if (SUMS_SMEM) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * sizeof(float) * S::CAP);
        if (e) return e;
    }
    return launch_pdl(kernel, dim3(p.blocks), dim3(S::THREADS), smem, s, p);
}

// The narrowest team that holds the row, 8 to 16 columns a thread: fewer threads per row
// means fewer barriers and more rows in flight per block.  16-byte units where every array
// is 16-byte aligned row by row, single elements otherwise.
template <typename T, typename W>
cudaError_t pick_fwd(const NormFwdParams& p, bool vec, cudaStream_t s) {
    constexpr int E = Elem<T>::VEC;
    const int w = p.width;
    if (vec) {
        if (w <= 8 * E) return run_fwd<T, W, true, 8, 1>(p, s);
        if (w <= 32 * E) return run_fwd<T, W, true, 32, 1>(p, s);
        if (w <= 512) return run_fwd<T, W, true, 32, 16 / E>(p, s);
        if (w <= 1024) return run_fwd<T, W, true, 128, 8 / E>(p, s);
        if (w <= 2048) return run_fwd<T, W, true, 128, 16 / E>(p, s);
        if (w <= 4096) return run_fwd<T, W, true, 256, 16 / E>(p, s);
        if (w <= 8192) return run_fwd<T, W, true, 512, 16 / E>(p, s);
        return run_fwd<T, W, true, 512, 32 / E>(p, s);
    }
    if (w <= 64) return run_fwd<T, W, false, 8, 8>(p, s);
    if (w <= 256) return run_fwd<T, W, false, 32, 8>(p, s);
    if (w <= 512) return run_fwd<T, W, false, 32, 16>(p, s);
    if (w <= 1024) return run_fwd<T, W, false, 128, 8>(p, s);
    if (w <= 2048) return run_fwd<T, W, false, 256, 8>(p, s);
    if (w <= 4096) return run_fwd<T, W, false, 512, 8>(p, s);
    if (w <= 8192) return run_fwd<T, W, false, 512, 16>(p, s);
    return run_fwd<T, W, false, 512, 32>(p, s);
}

template <typename T, typename W>
cudaError_t pick_bwd(const NormBwdParams& p, bool vec, cudaStream_t s) {
    constexpr int E = Elem<T>::VEC;
    const int w = p.width;
    if (vec) {
        if (w <= 8 * E) return run_bwd<T, W, true, 8, 1>(p, s);
        if (w <= 32 * E) return run_bwd<T, W, true, 32, 1>(p, s);
        if (w <= 512) return run_bwd<T, W, true, 32, 16 / E>(p, s);
        if (w <= 1024) return run_bwd<T, W, true, 128, 8 / E>(p, s);
        if (w <= 2048) return run_bwd<T, W, true, 128, 16 / E>(p, s);
        if (w <= 4096) return run_bwd<T, W, true, 256, 16 / E>(p, s);
        if (w <= 8192) return run_bwd<T, W, true, 512, 16 / E>(p, s);
        return run_bwd<T, W, true, 512, 32 / E, true>(p, s);
    }
    if (w <= 64) return run_bwd<T, W, false, 8, 8>(p, s);
    if (w <= 256) return run_bwd<T, W, false, 32, 8>(p, s);
    if (w <= 512) return run_bwd<T, W, false, 32, 16>(p, s);
    if (w <= 1024) return run_bwd<T, W, false, 128, 8>(p, s);
    if (w <= 2048) return run_bwd<T, W, false, 128, 16>(p, s);
    if (w <= 4096) return run_bwd<T, W, false, 256, 16>(p, s);
    if (w <= 8192) return run_bwd<T, W, false, 512, 16>(p, s);
    return run_bwd<T, W, false, 512, 32, true>(p, s);
}

}  // namespace

namespace {

// Threads of a team of the ring kernels: up to 16 columns each, off the 16-byte boundaries
// 8 where a block can hold that many threads twice.
// (2049 to 192 * 16 columns, forward, 192 threads against 256, us at 32768 rows: bf16 2056 columns
// 60/77, 2560 61/77, 2816 65/77, 3064 69/79; fp32 92/88, 110/120, 120/131, 131/140.  Backward 256 are
// faster, 2816 bf16 121 against 125.)
int ring_tpr(int width, int arrays, bool vec) {
    if (!vec && width <= 2048) return width <= 512 ? 64 : width <= 1024 ? 128 : 256;
    if (width <= 2048) return width <= 1024 ? 64 : 128;
    return width <= 192 * 16 && arrays == 1 ? 192 : width <= 4096 ? 256 : 512;
}

// Teams of the ring kernels on the whole device, and whether they run: two stages fit, rows
// too wide for a warp alone (off the 16-byte boundaries, backward only, 512 bytes), and enough
// rows per team to make up for a slower start.
// Measured with bf16, ring against plain, us: forward 768 columns 38.2/42.8 at 48 rows a team
// and 11.3/11.8 at 12, 1024 22.8/21.4 at 24, 2816 46.0/50.1 at 48 and 24.4/23.0 at 24; backward
// 2816 25.1/27.5 at 8 and 19.1/19.0 at 4; off the boundaries 500 columns 12.6/19.9 at 4, 1023
// 38.3/39.0 at 24 and 21.6/19.7 at 12, 2815 20.2/26.1 at 6; a warp for 512 columns against a ring
// of 32-thread teams 39.4/41.4 forward, 82/92 backward at 48.  (Forward one start for every width:
// 768 columns gain 4% at 12 rows already, 1024 and 2816 still lose 6% at 24.)
bool ring_plan(long long rows, int width, int dtype, bool vec, int arrays, int* blocks, int* team_rows) {
    const int es = dtype_size(dtype), tpr = ring_tpr(width, arrays, vec);
    const int least = arrays == 1 ? 32 : vec ? 8 : width <= 512 ? 4 : width <= 1024 ? 24 : 6;
    if ((vec ? width <= 512 : width * es < 512) || width > 8192) return false;
    if (ring_stages(tpr, arrays, ring_slot(vec, width * es)) < 2) return false;
    const int per_block = ring_teams(tpr);
    const long long teams = 152ll * ring_blocks(tpr) * per_block;
    if (rows < least * teams) return false;
    const long long each = (rows + teams - 1) / teams;
    *team_rows = static_cast<int>(each);
    *blocks = static_cast<int>((rows + each * per_block - 1) / (each * per_block));
    return true;
}

template <typename K, typename P>
cudaError_t run_ring(K kernel, const P& p, int tpr, int blocks, cudaStream_t s) {
    // All of a block's share of the shared memory, used or not: no SM takes one more block of the
    // next launch while this one's are leaving, which would leave another SM with one (32768 x
    // 2816 bf16 forward 91 us instead of 70).  The column sums reuse the ring.
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(tpr));
    if (e) return e;
    return launch_pdl(kernel, dim3(blocks), dim3(ring_threads(tpr)), ring_bytes(tpr), s, p);
}

template <typename T, typename W>
cudaError_t pick_fwd_ring(const NormFwdParams& p, int blocks, cudaStream_t s) {
    constexpr int NV = 16 / Elem<T>::VEC;
    const int tpr = ring_tpr(p.width, 1, true);
    switch (tpr) {
        case 64: return run_ring(norm_fwd_ring_kernel<T, W, 64, NV>, p, tpr, blocks, s);
        case 128: return run_ring(norm_fwd_ring_kernel<T, W, 128, NV>, p, tpr, blocks, s);
        case 192: return run_ring(norm_fwd_ring_kernel<T, W, 192, NV>, p, tpr, blocks, s);
        case 256: return run_ring(norm_fwd_ring_kernel<T, W, 256, NV>, p, tpr, blocks, s);
        default: return run_ring(norm_fwd_ring_kernel<T, W, 512, NV>, p, tpr, blocks, s);
    }
}
template <typename T, typename W>
cudaError_t pick_bwd_ring(const NormBwdParams& p, cudaStream_t s) {
    constexpr int NV = 16 / Elem<T>::VEC;
    const int arrays = p.res ? 3 : 2, tpr = ring_tpr(p.width, arrays, p.vec != 0);
    if (!p.vec) {
        switch (tpr) {
            case 64: return run_ring(norm_bwd_ring_kernel<T, W, false, 64, 8>, p, tpr, p.blocks, s);
            case 128: return run_ring(norm_bwd_ring_kernel<T, W, false, 128, 8>, p, tpr, p.blocks, s);
            case 256:
                return p.width <= 2048 ? run_ring(norm_bwd_ring_kernel<T, W, false, 256, 8>, p, tpr, p.blocks, s)
                                       : run_ring(norm_bwd_ring_kernel<T, W, false, 256, 16>, p, tpr, p.blocks, s);
            default: return run_ring(norm_bwd_ring_kernel<T, W, false, 512, 16>, p, tpr, p.blocks, s);
        }
    }
    switch (tpr) {
        case 64: return run_ring(norm_bwd_ring_kernel<T, W, true, 64, NV>, p, tpr, p.blocks, s);
        case 128: return run_ring(norm_bwd_ring_kernel<T, W, true, 128, NV>, p, tpr, p.blocks, s);
        case 256: return run_ring(norm_bwd_ring_kernel<T, W, true, 256, NV>, p, tpr, p.blocks, s);
        default: return run_ring(norm_bwd_ring_kernel<T, W, true, 512, NV>, p, tpr, p.blocks, s);
    }
}

template <typename T, typename W>
cudaError_t start_fwd(NormFwdParams p, bool vec, cudaStream_t s) {
    int blocks = 0;
    if (vec && ring_plan(p.rows, p.width, p.dtype, true, 1, &blocks, &p.team_rows)) return pick_fwd_ring<T, W>(p, blocks, s);
    return pick_fwd<T, W>(p, vec, s);
}
template <typename T, typename W>
cudaError_t start_bwd(const NormBwdParams& p, cudaStream_t s) {
    return p.team_rows ? pick_bwd_ring<T, W>(p, s) : pick_bwd<T, W>(p, p.vec != 0, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwdParams& p, cudaStream_t s) {
    const int es = dtype_size(p.dtype), ws = dtype_size(p.weight_dtype);
    const int unit = 16 / es;
    const bool vec = p.width % unit == 0 && aligned16(p.x, p.ldx, es, p.rows) && aligned16(p.y, p.ldy, es, p.rows) &&
                     aligned16(p.weight, 0, ws, 1) && aligned16(p.bias, 0, ws, 1);
    switch (p.dtype) {
        case DT_F32: return start_fwd<float, float>(p, vec, s);
        case DT_BF16:
            return p.weight_dtype == DT_F32 ? start_fwd<__nv_bfloat16, float>(p, vec, s)
                                            : start_fwd<__nv_bfloat16, __nv_bfloat16>(p, vec, s);
        default:
            return p.weight_dtype == DT_F32 ? start_fwd<__half, float>(p, vec, s) : start_fwd<__half, __half>(p, vec, s);
    }
}

static int plain_bwd_blocks(long long rows, int width) {
    // narrow rows: teams of 8 or 32 threads, 32 or 8 rows per block and turn; else one row
    // and a team of 128 threads or more, 16 columns of a row per thread
    const int per_block = width <= 64 ? 32 : width <= 512 ? 8 : 1;
    const int tpr = width <= 512 ? 32 : width <= 2048 ? 128 : width <= 4096 ? 256 : 512;
    const long long want = (rows + per_block - 1) / per_block;
    const long long cap = 152ll * bwd_blocks_per_sm(tpr);
    return static_cast<int>(want < 1 ? 1 : want < cap ? want : cap);
}

int norm_bwd_max_blocks(long long rows, int width, int dtype) {
    int most = plain_bwd_blocks(rows, width), blocks = 0, each = 0;
    for (int arrays = 2; arrays <= 3; ++arrays)
        for (int vec = 0; vec < 2; ++vec)
            if (ring_plan(rows, width, dtype, vec != 0, arrays, &blocks, &each) && blocks > most) most = blocks;
    return most;
}

void norm_bwd_plan(NormBwdParams* p) {
    const int es = dtype_size(p->dtype), ws = dtype_size(p->weight_dtype);
    const int unit = 16 / es;
    p->vec = p->width % unit == 0 && aligned16(p->x, p->ldx, es, p->rows) && aligned16(p->dy, p->lddy, es, p->rows) &&
             (!p->dx || aligned16(p->dx, p->lddx, es, p->rows)) && (!p->res || aligned16(p->res, p->ldr, es, p->rows)) &&
             aligned16(p->weight, 0, ws, 1);
    p->team_rows = 0;
    if (!ring_plan(p->rows, p->width, p->dtype, p->vec != 0, p->res ? 3 : 2, &p->blocks, &p->team_rows))
        p->blocks = plain_bwd_blocks(p->rows, p->width);
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, cudaStream_t s) {
    switch (p.dtype) {
        case DT_F32: return start_bwd<float, float>(p, s);
        case DT_BF16:
            return p.weight_dtype == DT_F32 ? start_bwd<__nv_bfloat16, float>(p, s)
                                            : start_bwd<__nv_bfloat16, __nv_bfloat16>(p, s);
        default: return p.weight_dtype == DT_F32 ? start_bwd<__half, float>(p, s) : start_bwd<__half, __half>(p, s);
    }
}

cudaError_t launch_norm_grads(const NormBwdParams& p, cudaStream_t s) {
    return launch_pdl(norm_grads_kernel, dim3((p.width + 31) / 32, 2), dim3(32 * GRAD_LANES), 0, s, p);
}

}  // namespace anvil
