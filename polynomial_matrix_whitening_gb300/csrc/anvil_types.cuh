// anvil_types.cuh -- the element types of the training-block operators (fp32, bf16, fp16):
// conversion to and from fp32 one by one and in 16-byte vectors, and the reductions over a
// team of threads.  Every sum is held in fp32; a value is rounded to its type once, as it
// is stored (round to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace anvil {

// dtype codes of include/anvil.h (anvil_dtype)
enum : int { DT_F32 = 0, DT_BF16 = 1, DT_F16 = 2 };
constexpr int dtype_size(int dt) { return dt == DT_F32 ? 4 : 2; }

// two fp32 in one 64-bit register pair
__device__ __forceinline__ uint64_t f2_make(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f2_split(uint64_t v, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int VEC = 4;  // elements in 16 bytes
    // a word of a very low value (-1e30, fp16: the lowest), and the word's values held to it
    // from below (NaN stays)
    static constexpr uint32_t LOW = 0xf1490000u;
    static __device__ __forceinline__ uint32_t not_below(uint32_t w) {
        uint32_t d;
        asm("max.NaN.f32 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(LOW));
        return d;
    }
    // the larger of two words' values, NaN ignored
    static __device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float word_max(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ float load(float v) { return v; }
    static __device__ __forceinline__ float store(float v) { return v; }
    static __device__ __forceinline__ void unpack(uint4 w, float* f) {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    // the same as packed fp32 pairs
    static __device__ __forceinline__ void unpack_pairs(uint4 w, uint64_t* p) {
        p[0] = f2_make(__uint_as_float(w.x), __uint_as_float(w.y));
        p[1] = f2_make(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ uint4 pack_pairs(const uint64_t* p) {
        float f[4];
        f2_split(p[0], f, f + 1);
        f2_split(p[1], f + 2, f + 3);
        return pack(f);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static constexpr uint32_t LOW = 0xf149f149u;
    static __device__ __forceinline__ uint32_t not_below(uint32_t w) {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(LOW));
        return d;
    }
    static __device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float word_max(uint32_t w) {
        return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ float load(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 store(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void unpack2(uint32_t w, float* f) {
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
        uint32_t d;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static __device__ __forceinline__ void unpack(uint4 w, float* f) {
        unpack2(w.x, f);
        unpack2(w.y, f + 2);
        unpack2(w.z, f + 4);
        unpack2(w.w, f + 6);
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
    static __device__ __forceinline__ uint64_t word_pair(uint32_t w) {
        float f[2];
        unpack2(w, f);
        return f2_make(f[0], f[1]);
    }
    static __device__ __forceinline__ uint32_t pair_word(uint64_t p) {
        float lo, hi;
        f2_split(p, &lo, &hi);
        return pack2(lo, hi);
    }
    static __device__ __forceinline__ void unpack_pairs(uint4 w, uint64_t* p) {
        p[0] = word_pair(w.x);
        p[1] = word_pair(w.y);
        p[2] = word_pair(w.z);
        p[3] = word_pair(w.w);
    }
    static __device__ __forceinline__ uint4 pack_pairs(const uint64_t* p) {
        return make_uint4(pair_word(p[0]), pair_word(p[1]), pair_word(p[2]), pair_word(p[3]));
    }
};
template <>
struct Elem<__half> {
    static constexpr int VEC = 8;
    static constexpr uint32_t LOW = 0xfbfffbffu;
    static __device__ __forceinline__ uint32_t not_below(uint32_t w) {
        uint32_t d;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(LOW));
        return d;
    }
    static __device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float word_max(uint32_t w) {
        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return fmaxf(r.x, r.y);
    }
    static __device__ __forceinline__ float load(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half store(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ void unpack2(uint32_t w, float* f) {
        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&w));
        f[0] = r.x;
        f[1] = r.y;
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ void unpack(uint4 w, float* f) {
        unpack2(w.x, f);
        unpack2(w.y, f + 2);
        unpack2(w.z, f + 4);
        unpack2(w.w, f + 6);
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
    static __device__ __forceinline__ uint64_t word_pair(uint32_t w) {
        float f[2];
        unpack2(w, f);
        return f2_make(f[0], f[1]);
    }
    static __device__ __forceinline__ uint32_t pair_word(uint64_t p) {
        float lo, hi;
        f2_split(p, &lo, &hi);
        return pack2(lo, hi);
    }
    static __device__ __forceinline__ void unpack_pairs(uint4 w, uint64_t* p) {
        p[0] = word_pair(w.x);
        p[1] = word_pair(w.y);
        p[2] = word_pair(w.z);
        p[3] = word_pair(w.w);
    }
    static __device__ __forceinline__ uint4 pack_pairs(const uint64_t* p) {
        return make_uint4(pair_word(p[0]), pair_word(p[1]), pair_word(p[2]), pair_word(p[3]));
    }
};

// (a.x b.x + c.x, a.y b.y + c.y) on packed fp32 pairs, one rounding each
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// Loads are the ordinary, coherent ones: a kernel that was launched early runs while the one ahead of
// it still writes, so nothing here is read-only for as long as the kernel runs (what __ldg asks for).
// Streaming 16-byte load (read once) and store (not read again soon).
__device__ __forceinline__ uint4 ldg_stream(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void stg_stream(void* p, uint4 v) { __stcs(reinterpret_cast<uint4*>(p), v); }

// Sum over a team of TPR consecutive threads (8 or 32: inside a warp; more: the whole
// block, through `red`, one float per warp).  Every thread of the team gets the same sum,
// in an order fixed by the thread numbers.  Callers alternate between arrays (16-byte
// aligned): one may be written again once every thread has passed another barrier.
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float* red) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; w += 4) {  // four warps' sums per load
            const float4 f = *reinterpret_cast<const float4*>(red + w);
            v += f.x;
            v += f.y;
            v += f.z;
            v += f.w;
        }
    }
    return v;
}

// Two sums at once (one barrier).
template <int TPR>
__device__ __forceinline__ void team_sum2(float& a, float& b, float2* red) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; w += 2) {  // two warps' sums per load
            const float4 f = *reinterpret_cast<const float4*>(red + w);
            a += f.x;
            b += f.y;
            a += f.z;
            b += f.w;
        }
    }
}

}  // namespace anvil
