// anvil_adamw.cu -- AdamW over many tensors in one launch, the moments in fp32 or in 8 bits.
//
//   g = grad grad_scale,  m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g g,
//   p = p decay - step_size m / (sqrt(v) root + eps)
// with step_size = lr / (1 - beta1^t), root = 1 / sqrt(1 - beta2^t), decay = 1 - lr weight_decay,
// fp32, one rounding per operation in the order written (no FMA).
//
// 8 bits.  256 consecutive values share an fp32 scale per moment, the block's largest magnitude
// over the largest code.  m is an e4m3 code (nearest, ties to even).  Of v the root r is kept, for
// two reasons: 8 bits of r span twice the range that they would span of v, and the step divides by
// r.  r >= 0 needs no sign, so its code c has four exponent and four fraction bits: c for c < 16,
// (16 + c % 16) 2^(c / 16 - 1) from there, up to 31 2^14: off by 2^-5 of itself at most over a
// range of 2^15 and reaching 2^19 down.  A root above 0 never becomes 0 (the code is at least 1): m / eps would
// follow where m's own code is not 0.  The step itself takes the unrounded moments.  A block whose
// largest magnitude is below 2^-100 is held as zeros; an infinity or a NaN makes its block NaN.
//
// What bounds it: HBM (28 bytes a value with everything in fp32, 16 with the states in 8 bits).
// A warp takes blocks of 256 values, a lane four neighbours at 4 lane and at 128 + 4 lane, so
// that every access of a warp is whole lines for 4-, 2- and 1-byte values alike; the block's
// largest magnitude is one redux over the values' bits, which puts NaN above all.  The tensors'
// pointers travel in the kernel's parameters (no table in device memory, so nothing is copied
// ahead and a captured graph holds everything); a thread block finds its tensor by bisection.
#include <cuda_runtime.h>
#include <stdint.h>

#include "anvil_adamw.h"
#include "anvil_device.cuh"
#include "anvil_types.cuh"

namespace anvil {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32, TURNS = ADAMW_CHUNK / (WARPS * ADAMW_BLOCK);
constexpr float TOP_M = 448.f, TOP_R = 507904.f;  // 31 2^14
constexpr float SMALLEST = 7.8886090522101181e-31f;  // 2^-100

// Eight values of a lane from an array of 4-, 2- or 1-byte elements, as their bits: four neighbours
// at a time, or one (what is at `left` and beyond reads as 0).
template <typename E>
__device__ __forceinline__ void load8(const E* p, bool vec, int lane, int left, E (&v)[8]) {
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const E* q = p + h * 128 + lane * 4;
            if constexpr (sizeof(E) == 4) {
                const uint4 w = __ldcs(reinterpret_cast<const uint4*>(q));
                v[4 * h] = w.x, v[4 * h + 1] = w.y, v[4 * h + 2] = w.z, v[4 * h + 3] = w.w;
            } else if constexpr (sizeof(E) == 2) {
                const uint2 w = __ldcs(reinterpret_cast<const uint2*>(q));
                v[4 * h] = w.x & 0xffffu, v[4 * h + 1] = w.x >> 16, v[4 * h + 2] = w.y & 0xffffu, v[4 * h + 3] = w.y >> 16;
            } else {
                const uint32_t w = __ldcs(reinterpret_cast<const uint32_t*>(q));
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * h + i] = (w >> 8 * i) & 0xffu;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i * 32 + lane < left ? __ldcs(p + i * 32 + lane) : E(0);
    }
}
template <typename E>
__device__ __forceinline__ void store8(E* p, bool vec, int lane, int left, const E (&v)[8]) {
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            E* q = p + h * 128 + lane * 4;
            const E* w = v + 4 * h;
            if constexpr (sizeof(E) == 4) {
                __stcs(reinterpret_cast<uint4*>(q), make_uint4(w[0], w[1], w[2], w[3]));
            } else if constexpr (sizeof(E) == 2) {
                __stcs(reinterpret_cast<uint2*>(q), make_uint2(w[0] | static_cast<uint32_t>(w[1]) << 16,
                                                               w[2] | static_cast<uint32_t>(w[3]) << 16));
            } else {
                __stcs(reinterpret_cast<uint32_t*>(q), w[0] | static_cast<uint32_t>(w[1]) << 8 |
                                                           static_cast<uint32_t>(w[2]) << 16 | static_cast<uint32_t>(w[3]) << 24);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane < left) __stcs(p + i * 32 + lane, v[i]);
    }
}

// The storage word of a type, and its value.
template <int DT>
struct Word;
template <>
struct Word<DT_F32> {
    using type = uint32_t;
    static __device__ __forceinline__ float value(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t word(float v) { return __float_as_uint(v); }
};
template <>
struct Word<DT_BF16> {
    using type = uint16_t;
    static __device__ __forceinline__ float value(uint16_t w) { return bf2f(w); }
    static __device__ __forceinline__ uint16_t word(float v) { return f2bf(v); }
};
template <>
struct Word<DT_F16> {
    using type = uint16_t;
    static __device__ __forceinline__ float value(uint16_t w) { return __half2float(__ushort_as_half(w)); }
    static __device__ __forceinline__ uint16_t word(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

__device__ __forceinline__ void e4m3_values(const uint8_t (&c)[8], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint16_t two = static_cast<uint16_t>(c[i] | c[i + 1] << 8);
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[i] = f.x;
        v[i + 1] = f.y;
    }
}
__device__ __forceinline__ void e4m3_codes(const float (&v)[8], uint8_t (&c)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(v[i + 1]), "f"(v[i]));
        c[i] = two & 0xff;
        c[i + 1] = two >> 8;
    }
}
// From 16 on the code's bits are the value's own: the exponent (less 130) and four fraction bits.
__device__ __forceinline__ float root_value(uint8_t c) {
    return c < 16 ? static_cast<float>(c) : __uint_as_float((static_cast<uint32_t>(c) << 19) + (130u << 23));
}
__device__ __forceinline__ uint8_t root_code(float q) {
    const uint32_t b = __float_as_uint(q);
    const int large = static_cast<int>((b + 0x3ffffu + (b >> 19 & 1u)) >> 19) - (131 << 4) + 16;
    const int c = q < 16.f ? __float2int_rn(q) : large;
    return static_cast<uint8_t>(q > 0.f ? min(max(c, 1), 255) : 0);
}

// A block's scale, and what its values are multiplied by for their codes.
struct Scale {
    float scale, inverse;
};
__device__ __forceinline__ Scale block_scale(const float (&v)[8], float top) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
    float f = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
    if (f < SMALLEST) f = 0.f;
    return {__fmul_rn(f, 1.f / top), f > 0.f ? __fdiv_rn(top, f) : 0.f};
}

// The tensor whose chunks hold `chunk`.
template <int N>
__device__ __forceinline__ int tensor_of(const AdamwParams<N>& a, int chunk) {
    int lo = 0, hi = a.tensors;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.t[mid].chunk0 <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int PARAM, int GRAD, bool CODES, int N>
__global__ void __launch_bounds__(THREADS) adamw_kernel(const __grid_constant__ AdamwParams<N> a) {
    constexpr bool SPLIT = PARAM == ADAMW_SPLIT;
    using P = Word<SPLIT ? DT_BF16 : PARAM>;
    using G = Word<GRAD>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AdamwTensor& t = a.t[tensor_of(a, blockIdx.x)];
    const long long blocks = (t.count + ADAMW_BLOCK - 1) / ADAMW_BLOCK;
    const long long first = static_cast<long long>(blockIdx.x - t.chunk0) * (ADAMW_CHUNK / ADAMW_BLOCK);
    pdl_allow_next();
    pdl_wait_previous();
    float step_size = a.scalars[0], root = a.scalars[1], decay = a.scalars[2], grad_scale = a.scalars[3];
    if (a.d_scalars) {
        step_size = a.d_scalars[0];
        root = a.d_scalars[1];
        decay = a.d_scalars[2];
        grad_scale = a.d_scalars[3];
    }
#pragma unroll 1
    for (int turn = 0; turn < TURNS; ++turn) {
        const long long b = first + turn * WARPS + warp;
        if (b >= blocks) break;
        const long long at = b * ADAMW_BLOCK;
        const int left = static_cast<int>(min(t.count - at, static_cast<long long>(ADAMW_BLOCK)));
        const bool vec = t.vec && left == ADAMW_BLOCK;
        typename P::type pw[8];
        typename G::type gw[8];
        uint16_t low[8];
        load8(static_cast<const typename P::type*>(t.p) + at, vec, lane, left, pw);
        if constexpr (SPLIT) load8(static_cast<const uint16_t*>(t.low) + at, vec, lane, left, low);
        load8(static_cast<const typename G::type*>(t.g) + at, vec, lane, left, gw);
        float m[8], v[8], r[8];
        if constexpr (CODES) {
            uint8_t mc[8], vc[8];
            load8(static_cast<const uint8_t*>(t.m) + at, vec, lane, left, mc);
            load8(static_cast<const uint8_t*>(t.v) + at, vec, lane, left, vc);
            const float ms = t.scales[b], rs = t.scales[blocks + b];
            e4m3_values(mc, m);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = __fmul_rn(m[i], ms);
                const float root0 = __fmul_rn(root_value(vc[i]), rs);
                v[i] = __fmul_rn(root0, root0);
            }
        } else {
            uint32_t w[8];
            load8(static_cast<const uint32_t*>(t.m) + at, vec, lane, left, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = __uint_as_float(w[i]);
            load8(static_cast<const uint32_t*>(t.v) + at, vec, lane, left, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float g = __fmul_rn(G::value(gw[i]), grad_scale);
            m[i] = __fadd_rn(__fmul_rn(m[i], a.beta1), __fmul_rn(g, a.c1));
            v[i] = __fadd_rn(__fmul_rn(v[i], a.beta2), __fmul_rn(__fmul_rn(g, a.c2), g));
            r[i] = __fsqrt_rn(v[i]);
            const float u = __fmul_rn(__fdiv_rn(m[i], __fadd_rn(__fmul_rn(r[i], root), a.eps)), step_size);
            float p;
            if constexpr (SPLIT) p = __uint_as_float(static_cast<uint32_t>(pw[i]) << 16 | low[i]);
            else p = P::value(pw[i]);
            p = __fsub_rn(__fmul_rn(p, decay), u);
            if constexpr (SPLIT) {
                const uint32_t bits = __float_as_uint(p);
                pw[i] = bits >> 16;
                low[i] = bits & 0xffffu;
            } else {
                pw[i] = P::word(p);
            }
        }
        store8(static_cast<typename P::type*>(t.p) + at, vec, lane, left, pw);
        if constexpr (SPLIT) store8(t.low + at, vec, lane, left, low);
        if constexpr (CODES) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!vec && i * 32 + lane >= left) m[i] = r[i] = 0.f;  // behind the tensor's end
            const Scale sm = block_scale(m, TOP_M), sr = block_scale(r, TOP_R);
            uint8_t c[8];
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(m[i], sm.inverse);
            e4m3_codes(q, c);
            store8(static_cast<uint8_t*>(t.m) + at, vec, lane, left, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = root_code(__fmul_rn(r[i], sr.inverse));
            store8(static_cast<uint8_t*>(t.v) + at, vec, lane, left, c);
            if (lane == 0) {
                t.scales[b] = sm.scale;
                t.scales[blocks + b] = sr.scale;
            }
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(m[i]);
            store8(static_cast<uint32_t*>(t.m) + at, vec, lane, left, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
            store8(static_cast<uint32_t*>(t.v) + at, vec, lane, left, w);
        }
    }
}

// What the codes stand for (10 bytes a value: HBM).
template <int N>
__global__ void __launch_bounds__(THREADS) adamw_values_kernel(const __grid_constant__ AdamwParams<N> a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AdamwTensor& t = a.t[tensor_of(a, blockIdx.x)];
    const long long blocks = (t.count + ADAMW_BLOCK - 1) / ADAMW_BLOCK;
    const long long first = static_cast<long long>(blockIdx.x - t.chunk0) * (ADAMW_CHUNK / ADAMW_BLOCK);
    pdl_allow_next();
    pdl_wait_previous();
#pragma unroll
    for (int turn = 0; turn < TURNS; ++turn) {
        const long long b = first + turn * WARPS + warp;
        if (b >= blocks) break;
        const long long at = b * ADAMW_BLOCK;
        const int left = static_cast<int>(min(t.count - at, static_cast<long long>(ADAMW_BLOCK)));
        const bool vec = t.vec && left == ADAMW_BLOCK;
        uint8_t mc[8], vc[8];
        load8(static_cast<const uint8_t*>(t.m) + at, vec, lane, left, mc);
        load8(static_cast<const uint8_t*>(t.v) + at, vec, lane, left, vc);
        const float ms = t.scales[b], rs = t.scales[blocks + b];
        float m[8];
        uint32_t w[8];
        e4m3_values(mc, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__fmul_rn(m[i], ms));
        store8(static_cast<uint32_t*>(t.p) + at, vec, lane, left, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = __fmul_rn(root_value(vc[i]), rs);
            w[i] = __float_as_uint(__fmul_rn(r, r));
        }
        store8(static_cast<uint32_t*>(const_cast<void*>(t.g)) + at, vec, lane, left, w);
    }
}

// A launch's parameters by the room that they need: 30 KB of them take the host and the device
// longer than a few tensors' work.
AdamwParams<ADAMW_FEW> few_of(const AdamwGroup& g) {
    AdamwParams<ADAMW_FEW> p;
    for (int i = 0; i < g.p.tensors; ++i) p.t[i] = g.p.t[i];
    p.tensors = g.p.tensors;
    p.beta1 = g.p.beta1;
    p.c1 = g.p.c1;
    p.beta2 = g.p.beta2;
    p.c2 = g.p.c2;
    p.eps = g.p.eps;
    for (int i = 0; i < 4; ++i) p.scalars[i] = g.p.scalars[i];
    p.d_scalars = g.p.d_scalars;
    return p;
}

template <int PARAM, int GRAD, bool CODES>
cudaError_t run(const AdamwGroup& g, cudaStream_t s) {
    if (g.p.tensors <= ADAMW_FEW)
        return launch_pdl(adamw_kernel<PARAM, GRAD, CODES, ADAMW_FEW>, dim3(g.chunks), dim3(THREADS), 0, s, few_of(g));
    return launch_pdl(adamw_kernel<PARAM, GRAD, CODES, ADAMW_MANY>, dim3(g.chunks), dim3(THREADS), 0, s, g.p);
}
template <int PARAM, int GRAD>
cudaError_t pick(const AdamwGroup& g, bool codes, cudaStream_t s) {
    return codes ? run<PARAM, GRAD, true>(g, s) : run<PARAM, GRAD, false>(g, s);
}

}  // namespace

cudaError_t launch_adamw(const AdamwGroup& g, int param, int grad, bool codes, cudaStream_t s) {
    switch (param * 4 + grad) {
        case ADAMW_F32 * 4 + DT_F32: return pick<ADAMW_F32, DT_F32>(g, codes, s);
        case ADAMW_F32 * 4 + DT_BF16: return pick<ADAMW_F32, DT_BF16>(g, codes, s);
        case ADAMW_F32 * 4 + DT_F16: return pick<ADAMW_F32, DT_F16>(g, codes, s);
        case ADAMW_BF16 * 4 + DT_F32: return pick<ADAMW_BF16, DT_F32>(g, codes, s);
        case ADAMW_BF16 * 4 + DT_BF16: return pick<ADAMW_BF16, DT_BF16>(g, codes, s);
        case ADAMW_F16 * 4 + DT_F32: return pick<ADAMW_F16, DT_F32>(g, codes, s);
        case ADAMW_F16 * 4 + DT_F16: return pick<ADAMW_F16, DT_F16>(g, codes, s);
        case ADAMW_SPLIT * 4 + DT_F32: return pick<ADAMW_SPLIT, DT_F32>(g, codes, s);
        case ADAMW_SPLIT * 4 + DT_BF16: return pick<ADAMW_SPLIT, DT_BF16>(g, codes, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_adamw_values(const AdamwGroup& g, cudaStream_t s) {
    if (g.p.tensors <= ADAMW_FEW)
        return launch_pdl(adamw_values_kernel<ADAMW_FEW>, dim3(g.chunks), dim3(THREADS), 0, s, few_of(g));
    return launch_pdl(adamw_values_kernel<ADAMW_MANY>, dim3(g.chunks), dim3(THREADS), 0, s, g.p);
}

}  // namespace anvil
