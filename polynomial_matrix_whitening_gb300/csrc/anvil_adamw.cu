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

#include <type_traits>

#include "anvil_adamw.h"
#include "anvil_device.cuh"
#include "anvil_round.cuh"
#include "anvil_types.cuh"

namespace anvil {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr float TOP_M = 448.f, TOP_R = 507904.f;  // 31 2^14
constexpr float SMALLEST = 7.8886090522101181e-31f;  // 2^-100

// Eight values of a lane from an array of 4-, 2- or 1-byte elements, as they were loaded: nothing
// uses them before they are needed, so a block's loads are on their way while the one before it is
// computed.  VEC: whole blocks are on vector boundaries, four neighbours at a time.  Otherwise,
// and in a tensor's last block (not WHOLE), one by one (what is at `left` and beyond reads as 0).
template <typename E, bool VEC>
struct Eight {
    static constexpr int W = VEC ? 2 * sizeof(E) : 8;  // words
    uint32_t w[W];
    template <bool WHOLE>
    __device__ __forceinline__ void load(const E* p, int lane, int left) {
        if constexpr (VEC && WHOLE) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const E* q = p + h * 128 + lane * 4;
                if constexpr (sizeof(E) == 4) {
                    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(q));
                    w[4 * h] = x.x, w[4 * h + 1] = x.y, w[4 * h + 2] = x.z, w[4 * h + 3] = x.w;
                } else if constexpr (sizeof(E) == 2) {
                    const uint2 x = __ldcs(reinterpret_cast<const uint2*>(q));
                    w[2 * h] = x.x, w[2 * h + 1] = x.y;
                } else {
                    w[h] = __ldcs(reinterpret_cast<const uint32_t*>(q));
                }
            }
            return;
        }
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t x = WHOLE || i * 32 + lane < left ? static_cast<uint32_t>(__ldcs(p + i * 32 + lane)) : 0u;
            if constexpr (VEC) w[i * sizeof(E) / 4] |= x << (i * sizeof(E) % 4 * 8);
            else w[i] = x;
        }
    }
    __device__ __forceinline__ E operator[](int i) const {
        if constexpr (VEC) return static_cast<E>(w[i * sizeof(E) / 4] >> (i * sizeof(E) % 4 * 8));
        else return static_cast<E>(w[i]);
    }
};
template <bool VEC, bool WHOLE, typename E>
__device__ __forceinline__ void store8(E* p, int lane, int left, const E (&v)[8]) {
    if constexpr (VEC && WHOLE) {
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
            if (WHOLE || i * 32 + lane < left) __stcs(p + i * 32 + lane, v[i]);
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

template <bool VEC>
__device__ __forceinline__ void e4m3_values(const Eight<uint8_t, VEC>& c, float (&v)[8]) {
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
// A root's code is an fp16 number's exponent (its lower four bits) and first four fraction bits, 0 to 15
// its subnormal ones: shifted there it is the value over 2^18.
template <bool VEC>
__device__ __forceinline__ void root_values(const Eight<uint8_t, VEC>& c, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint32_t h;
        if constexpr (VEC) h = __byte_perm(c.w[i / 4], 0, i % 4 ? 0x4342 : 0x4140) << 6;
        else h = (c.w[i] | c.w[i + 1] << 16) << 6;
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[i] = f.x;
        v[i + 1] = f.y;
    }
}
constexpr float ROOT_UNIT = 262144.f;  // 2^18
// The nearest code of q (507904 at most, but for its rounding), ties to the even one: adding 2^19 times
// the power of two below q (16 at least) leaves q's first five bits, rounded, at the end of the sum.  A q
// above 0 has a code of 1 at least; NaN gives 0.  Only the low byte counts.
__device__ __forceinline__ uint32_t root_code(float q) {
    const uint32_t power = max(__float_as_uint(q) & 0x7f800000u, 131u << 23);
    const uint32_t sum = __float_as_uint(__fadd_rn(q, __uint_as_float(power + (19u << 23))));
    const uint32_t c = ((power >> 19) + sum - (131u << 4)) & 0xffu;
    return q > 0.f ? max(c, 1u) : 0u;
}

// The largest of a lane's values (magnitudes: bits without the sign), as bits, which puts an infinity
// above every number and a NaN above that.
template <bool SIGNED>
__device__ __forceinline__ uint32_t most_bits(const float (&v)[8]) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, SIGNED ? __float_as_uint(v[i]) & 0x7fffffffu : __float_as_uint(v[i]));
    return most;
}

// The least magnitude of a lane's values that are not 0, as bits less 1, which puts 0 above all.
__device__ __forceinline__ uint32_t least_bits(const float (&v)[8]) {
    uint32_t least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 8; ++i) least = min(least, (__float_as_uint(v[i]) & 0x7fffffffu) - 1u);
    return least;
}

// The eight values times one factor, in pairs.
__device__ __forceinline__ void times8(float (&v)[8], float f) {
    const uint64_t ff = f2_make(f, f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) f2_split(f2_mul(f2_make(v[i], v[i + 1]), ff), &v[i], &v[i + 1]);
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

// What a block's step reads.
template <int PARAM, int GRAD, bool CODES, bool VEC>
struct Inputs {
    static constexpr bool SPLIT = PARAM == ADAMW_SPLIT;
    using P = Word<SPLIT ? DT_BF16 : PARAM>;
    using G = Word<GRAD>;
    using S = std::conditional_t<CODES, uint8_t, uint32_t>;
    Eight<typename P::type, VEC> p;
    Eight<uint16_t, VEC> low;
    Eight<typename G::type, VEC> g;
    Eight<S, VEC> m, v;
    float ms, rs;
    // gradient and moments, and the parameter: apart, since they are used at different times
    template <bool WHOLE>
    __device__ __forceinline__ void load_moments(const AdamwTensor& t, long long block, long long blocks, int lane) {
        const long long at = block * ADAMW_BLOCK;
        const int left = WHOLE ? ADAMW_BLOCK : static_cast<int>(t.count - at);
        g.template load<WHOLE>(static_cast<const typename G::type*>(t.g) + at, lane, left);
        m.template load<WHOLE>(static_cast<const S*>(t.m) + at, lane, left);
        v.template load<WHOLE>(static_cast<const S*>(t.v) + at, lane, left);
        if constexpr (CODES) {
            ms = t.scales[block];
            rs = t.scales[blocks + block];
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ void load_param(const AdamwTensor& t, long long block, int lane) {
        const long long at = block * ADAMW_BLOCK;
        const int left = WHOLE ? ADAMW_BLOCK : static_cast<int>(t.count - at);
        p.template load<WHOLE>(static_cast<const typename P::type*>(t.p) + at, lane, left);
        if constexpr (SPLIT) low.template load<WHOLE>(t.low + at, lane, left);
    }
};
struct Constants {
    float beta1, c1, beta2, c2, eps, step_size, root, decay, grad_scale;
    bool middle;  // denominators from 2^-60 (eps) to 2^24 (2^13 2^10 + eps)
};

// One block's step from what `in` holds; as soon as that is used, what block `next` (whole; -1: none) needs
// takes its place.
template <int PARAM, int GRAD, bool CODES, bool VEC, bool WHOLE>
__device__ __forceinline__ void adamw_block(const AdamwTensor& t, const Constants& a, Inputs<PARAM, GRAD, CODES, VEC>& in, long long b,
                                            long long next, long long blocks, int lane) {
    using In = Inputs<PARAM, GRAD, CODES, VEC>;
    using P = typename In::P;
    using G = typename In::G;
    constexpr bool SPLIT = In::SPLIT;
    const long long at = b * ADAMW_BLOCK;
    const int left = WHOLE ? ADAMW_BLOCK : static_cast<int>(t.count - at);
    float m[8], v[8], r[8], u[8];
    if constexpr (CODES) {
        e4m3_values(in.m, m);
        times8(m, in.ms);
        root_values(in.v, v);
        times8(v, __fmul_rn(in.rs, ROOT_UNIT));
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint64_t x = f2_make(v[i], v[i + 1]);
            f2_split(f2_mul(x, x), &v[i], &v[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = __uint_as_float(in.m[i]);
            v[i] = __uint_as_float(in.v[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float g = __fmul_rn(G::value(in.g[i]), a.grad_scale);
        m[i] = __fadd_rn(__fmul_rn(m[i], a.beta1), __fmul_rn(g, a.c1));
        v[i] = __fadd_rn(__fmul_rn(v[i], a.beta2), __fmul_rn(__fmul_rn(g, a.c2), g));
    }
    if (next >= 0) in.template load_moments<true>(t, next, blocks, lane);
    if constexpr (CODES && !WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane >= left) m[i] = v[i] = 0.f;  // behind the tensor's end
    }
    uint32_t most_m = 0, most_v = 0;
    if constexpr (CODES) {
        most_m = most_bits<true>(m);
        most_v = most_bits<false>(v);
    }
    // |m| 0 or from 2^-102 (no quotient below 2^-126, and every remainder exact) to 2^60 (none overflows) and v below
    // 2^26, no infinity or NaN among them
    if (CODES && a.middle && least_bits(m) >= (25u << 23) - 1u && most_m < (187u << 23) && most_v < (153u << 23)) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            f2_split(f2_root(f2_make(v[i], v[i + 1])), &r[i], &r[i + 1]);
            const uint64_t d = f2_make(__fadd_rn(__fmul_rn(r[i], a.root), a.eps), __fadd_rn(__fmul_rn(r[i + 1], a.root), a.eps));
            f2_split(f2_divide(f2_make(m[i], m[i + 1]), d), &u[i], &u[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] = __fsqrt_rn(v[i]);
            u[i] = __fdiv_rn(m[i], __fadd_rn(__fmul_rn(r[i], a.root), a.eps));
        }
    }
    typename P::type pw[8];
    uint16_t low[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float p;
        if constexpr (SPLIT) p = __uint_as_float(static_cast<uint32_t>(in.p[i]) << 16 | in.low[i]);
        else p = P::value(in.p[i]);
        p = __fsub_rn(__fmul_rn(p, a.decay), __fmul_rn(u[i], a.step_size));
        if constexpr (SPLIT) {
            const uint32_t bits = __float_as_uint(p);
            pw[i] = bits >> 16;
            low[i] = bits & 0xffffu;
        } else {
            pw[i] = P::word(p);
        }
    }
    if (next >= 0) in.template load_param<true>(t, next, lane);
    store8<VEC, WHOLE>(static_cast<typename P::type*>(t.p) + at, lane, left, pw);
    if constexpr (SPLIT) store8<VEC, WHOLE>(t.low + at, lane, left, low);
    if constexpr (CODES) {
        // the scales (the largest root is the largest v's), and what the values are multiplied by for their codes
        most_m = __reduce_max_sync(0xffffffffu, most_m);
        most_v = __reduce_max_sync(0xffffffffu, most_v);
        float fm = __uint_as_float(most_m), fr, im, ir;
        // |m| and v where the pair's root and quotients reach (the same for the whole warp)
        if (most_m >= (67u << 23) && most_m < (187u << 23) && most_v >= (37u << 23) && most_v < (153u << 23)) {
            float other;
            f2_split(f2_root(f2_make(__uint_as_float(most_v), 0.f)), &fr, &other);
            f2_split(f2_divide(f2_make(TOP_M, TOP_R), f2_make(fm, fr)), &im, &ir);
        } else {
            fr = __fsqrt_rn(__uint_as_float(most_v));
            if (fm < SMALLEST) fm = 0.f;
            if (fr < SMALLEST) fr = 0.f;
            im = fm > 0.f ? __fdiv_rn(TOP_M, fm) : 0.f;
            ir = fr > 0.f ? __fdiv_rn(TOP_R, fr) : 0.f;
        }
        if (lane < 2) t.scales[lane ? blocks + b : b] = lane ? __fmul_rn(fr, 1.f / TOP_R) : __fmul_rn(fm, 1.f / TOP_M);
        uint8_t c[8];
        times8(m, im);
        e4m3_codes(m, c);
        store8<VEC, WHOLE>(static_cast<uint8_t*>(t.m) + at, lane, left, c);
        times8(r, ir);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = static_cast<uint8_t>(root_code(r[i]));
        store8<VEC, WHOLE>(static_cast<uint8_t*>(t.v) + at, lane, left, c);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(m[i]);
        store8<VEC, WHOLE>(static_cast<uint32_t*>(t.m) + at, lane, left, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
        store8<VEC, WHOLE>(static_cast<uint32_t*>(t.v) + at, lane, left, w);
    }
}

// With fp32 states the kernel waits for memory (50M split bf16 values 190 us, 6.8 TB/s).  With codes it is
// short of instructions (98 a value, at 80% of the issue slots, in its first form): quotients and roots
// there are pairs without the general ones' branches (where a lane's values are in the middle of the
// range), and a tensor's last block, the only one with bounds, is apart.  134M fp32 values: 470 us in the
// first form, 365 now (5.9 TB/s); four blocks an SM, three where their registers are needed (with codes 3 gives 405).
template <int PARAM, int GRAD, bool CODES, bool VEC, int N>
__global__ void __launch_bounds__(THREADS, CODES && VEC ? 4 : 3) adamw_kernel(const __grid_constant__ AdamwParams<N> p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AdamwTensor& t = p.t[tensor_of(p, blockIdx.x)];
    const long long blocks = (t.count + ADAMW_BLOCK - 1) / ADAMW_BLOCK;
    const long long first = static_cast<long long>(blockIdx.x - t.chunk0) * p.chunk, end = min(blocks, first + p.chunk);
    const long long whole = min(t.count / ADAMW_BLOCK, end);
    pdl_allow_next();
    pdl_wait_previous();
    Constants a = {p.beta1, p.c1, p.beta2, p.c2, p.eps, p.scalars[0], p.scalars[1], p.scalars[2], p.scalars[3], false};
    if (p.d_scalars) {
        a.step_size = p.d_scalars[0];
        a.root = p.d_scalars[1];
        a.decay = p.d_scalars[2];
        a.grad_scale = p.d_scalars[3];
    }
    a.middle = a.eps >= 0x1p-60f && a.eps <= 1.f && a.root >= 0.f && a.root <= 0x1p10f;
    Inputs<PARAM, GRAD, CODES, VEC> in;
    long long b = first + warp;
    if (b < whole) {
        in.template load_moments<true>(t, b, blocks, lane);
        in.template load_param<true>(t, b, lane);
    }
#pragma unroll 1
    for (; b < whole; b += WARPS) adamw_block<PARAM, GRAD, CODES, VEC, true>(t, a, in, b, b + WARPS < whole ? b + WARPS : -1, blocks, lane);
    if (b < end) {  // the block behind the whole ones
        in.template load_moments<false>(t, b, blocks, lane);
        in.template load_param<false>(t, b, lane);
        adamw_block<PARAM, GRAD, CODES, VEC, false>(t, a, in, b, -1, blocks, lane);
    }
}

// What the codes stand for (10 bytes a value: HBM).
template <bool VEC, int N>
__global__ void __launch_bounds__(THREADS) adamw_values_kernel(const __grid_constant__ AdamwParams<N> a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AdamwTensor& t = a.t[tensor_of(a, blockIdx.x)];
    const long long blocks = (t.count + ADAMW_BLOCK - 1) / ADAMW_BLOCK;
    const long long first = static_cast<long long>(blockIdx.x - t.chunk0) * a.chunk, end = min(blocks, first + a.chunk);
    pdl_allow_next();
    pdl_wait_previous();
    const long long whole = min(t.count / ADAMW_BLOCK, end);
    struct In {
        Eight<uint8_t, VEC> m, v;
        float ms, rs;
    } now, next;
    const auto load = [&](auto is_whole, long long b, In& in) {
        constexpr bool WHOLE = decltype(is_whole)::value;
        const long long at = b * ADAMW_BLOCK;
        in.m.template load<WHOLE>(static_cast<const uint8_t*>(t.m) + at, lane, static_cast<int>(t.count - at));
        in.v.template load<WHOLE>(static_cast<const uint8_t*>(t.v) + at, lane, static_cast<int>(t.count - at));
        in.ms = t.scales[b];
        in.rs = t.scales[blocks + b];
    };
    const auto send = [&](auto is_whole, long long b, const In& in) {
        constexpr bool WHOLE = decltype(is_whole)::value;
        const long long at = b * ADAMW_BLOCK;
        const int left = static_cast<int>(t.count - at);
        float m[8];
        uint32_t w[8];
        e4m3_values(in.m, m);
        times8(m, in.ms);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(m[i]);
        store8<VEC, WHOLE>(static_cast<uint32_t*>(t.p) + at, lane, left, w);
        root_values(in.v, m);
        times8(m, __fmul_rn(in.rs, ROOT_UNIT));
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__fmul_rn(m[i], m[i]));
        store8<VEC, WHOLE>(static_cast<uint32_t*>(const_cast<void*>(t.g)) + at, lane, left, w);
    };
    long long b = first + warp;
    if (b < whole) load(std::true_type(), b, next);
#pragma unroll 1
    for (; b < whole; b += WARPS) {
        now = next;
        if (b + WARPS < whole) load(std::true_type(), b + WARPS, next);
        send(std::true_type(), b, now);
    }
    if (b < end) {
        load(std::false_type(), b, now);
        send(std::false_type(), b, now);
    }
}

// A launch's parameters by the room that they need: 30 KB of them take the host and the device
// longer than a few tensors' work.
AdamwParams<ADAMW_FEW> few_of(const AdamwGroup& g) {
    AdamwParams<ADAMW_FEW> p;
    for (int i = 0; i < g.p.tensors; ++i) p.t[i] = g.p.t[i];
    p.tensors = g.p.tensors;
    p.chunk = g.p.chunk;
    p.beta1 = g.p.beta1;
    p.c1 = g.p.c1;
    p.beta2 = g.p.beta2;
    p.c2 = g.p.c2;
    p.eps = g.p.eps;
    for (int i = 0; i < 4; ++i) p.scalars[i] = g.p.scalars[i];
    p.d_scalars = g.p.d_scalars;
    return p;
}

template <int PARAM, int GRAD, bool CODES, bool VEC>
cudaError_t run(const AdamwGroup& g, cudaStream_t s) {
    const dim3 grid(g.chunks), block(THREADS);
    if (g.p.tensors <= ADAMW_FEW) return launch_pdl(adamw_kernel<PARAM, GRAD, CODES, VEC, ADAMW_FEW>, grid, block, 0, s, few_of(g));
    return launch_pdl(adamw_kernel<PARAM, GRAD, CODES, VEC, ADAMW_MANY>, grid, block, 0, s, g.p);
}
template <int PARAM, int GRAD>
cudaError_t pick(const AdamwGroup& g, bool codes, bool vec, cudaStream_t s) {
    if (codes) return vec ? run<PARAM, GRAD, true, true>(g, s) : run<PARAM, GRAD, true, false>(g, s);
    return vec ? run<PARAM, GRAD, false, true>(g, s) : run<PARAM, GRAD, false, false>(g, s);
}
template <bool VEC>
cudaError_t run_values(const AdamwGroup& g, cudaStream_t s) {
    const dim3 grid(g.chunks), block(THREADS);
    if (g.p.tensors <= ADAMW_FEW) return launch_pdl(adamw_values_kernel<VEC, ADAMW_FEW>, grid, block, 0, s, few_of(g));
    return launch_pdl(adamw_values_kernel<VEC, ADAMW_MANY>, grid, block, 0, s, g.p);
}

}  // namespace

cudaError_t launch_adamw(const AdamwGroup& g, int param, int grad, bool codes, bool vec, cudaStream_t s) {
    switch (param * 4 + grad) {
        case ADAMW_F32 * 4 + DT_F32: return pick<ADAMW_F32, DT_F32>(g, codes, vec, s);
        case ADAMW_F32 * 4 + DT_BF16: return pick<ADAMW_F32, DT_BF16>(g, codes, vec, s);
        case ADAMW_F32 * 4 + DT_F16: return pick<ADAMW_F32, DT_F16>(g, codes, vec, s);
        case ADAMW_BF16 * 4 + DT_F32: return pick<ADAMW_BF16, DT_F32>(g, codes, vec, s);
        case ADAMW_BF16 * 4 + DT_BF16: return pick<ADAMW_BF16, DT_BF16>(g, codes, vec, s);
        case ADAMW_F16 * 4 + DT_F32: return pick<ADAMW_F16, DT_F32>(g, codes, vec, s);
        case ADAMW_F16 * 4 + DT_F16: return pick<ADAMW_F16, DT_F16>(g, codes, vec, s);
        case ADAMW_SPLIT * 4 + DT_F32: return pick<ADAMW_SPLIT, DT_F32>(g, codes, vec, s);
        case ADAMW_SPLIT * 4 + DT_BF16: return pick<ADAMW_SPLIT, DT_BF16>(g, codes, vec, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_adamw_values(const AdamwGroup& g, bool vec, cudaStream_t s) {
    return vec ? run_values<true>(g, s) : run_values<false>(g, s);
}

}  // namespace anvil
