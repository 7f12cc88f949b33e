// anvil_logprob.cu -- log probabilities of given tokens, with entropy and the top
// alternatives, and their gradient, for sm_103a.
//
//   forward   lse = log sum_j e^{x_j},  logprob = x_t - lse,  H = lse - sum_j p_j x_j,
//             the k largest x_j - lse (ties: the lowest index first), p_j = e^{x_j - lse}
//   backward  dx_j = u ([j = t] - p_j) - v p_j (log p_j + H)
//             for u = dL/dlogprob, v = dL/dH
//
// The forward pass reads the logits once: every thread keeps a running maximum m, the sum
// s of e^{x - m} and the sum q of e^{x - m} (x - m) (in fp32, rescaled when the maximum
// grows), from which lse = m + log s and H = log s - q / s.  The arithmetic runs on packed
// fp32 pairs: about 4.5 instructions per element, where scalar ones took 8 and the issue
// rate, not HBM, was the bound.
//
// The top k cost the pass one store a turn: every thread keeps the largest of its values of
// each turn (32 values, fp32: 16) in shared memory.  The k-th largest of the 32 lanes' maxima
// (over the warps) is a value that at least k elements reach, and hardly more do; the few
// turns whose maximum reaches it are read again (from L2), their elements that reach it are
// listed, and the entries ahead of each are counted: its place.  Where more elements reach it
// than the list holds (many equal values, a masked row), the larger ones are listed and the
// first of the equal ones; where the larger ones alone are too many (they share a few lanes),
// every warp walks its elements in order and keeps the best k, one per lane.
//
// HBM bounds both passes where there are many rows; where rows are fewer than the SMs, a
// cluster of up to eight blocks takes a row's segments and the first block joins their
// results through distributed shared memory, in a fixed order.
//
// A row in which every logit is -inf has no distribution: lse and the log probabilities
// are -inf, the entropy is 0 and the gradient is zero.  A masked logit (-inf, or the type's
// lowest value) adds nothing: the forward pass takes values below -1e30 as that (fp16: -inf as
// the lowest value), which keeps e y = 0 without a test; a row whose maximum, or whose k-th
// value, is not far above that is taken again value by value.  The gradient, where a vector's
// sum of e y comes out NaN, from 0 times infinity, takes the vector again with the exponents
// held at -200 (in base 2), where e is 0.  A NaN or +inf makes its row NaN.
//
// The exponentials flush results below 2^-126 to 0 (keeping them takes three more instructions an
// element): a sum does not see them, a gradient loses what is under 1e-36 of u and v.
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "anvil_device.cuh"
#include "anvil_internal.h"
#include "anvil_logprob.h"
#include "anvil_types.cuh"

namespace anvil {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr int KEY_NONE = INT32_MIN;  // below every key of a value

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}

// Running statistics: maximum m, s = sum 2^{y}, q = sum 2^{y} y with y = (x - m) log2 e.
struct Stats {
    float m, s, q;
};
// Statistics over a larger maximum.
__device__ __forceinline__ Stats over(Stats a, float m) {
    const float d = fmaxf((a.m - (m == -INFINITY ? 0.f : m)) * LOG2E, -200.f), c = ex2(d);
    a.q = c * (a.q + d * a.s);
    a.s *= c;
    a.m = m;
    return a;
}
// The statistics of W lanes together, in every one of them: one rescaling to their common
// maximum, then plain sums.  Empty lanes have m = -inf, s = q = 0.
template <int W>
__device__ __forceinline__ Stats join(Stats a) {
    float m = a.m;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    a = over(a, m);
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        a.q += __shfl_xor_sync(0xffffffffu, a.q, o);
    }
    return a;
}

// Order of the alternatives: larger value first, then lower index.  Floats compare as the
// integers of their order (-0 as +0).
__device__ __forceinline__ int order_key(float v) {
    const int b = __float_as_int(v + 0.f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }
__device__ __forceinline__ bool better(int ka, int ia, int kb, int ib) { return ka > kb || (ka == kb && ia < ib); }

// A warp's list of its best `top` entries: lane l holds the l-th.
struct TopList {
    int key, idx;  // this lane's entry
    int kth_key, kth_idx;
};
__device__ __forceinline__ void top_init(TopList& L) {
    L.key = L.kth_key = KEY_NONE;
    L.idx = L.kth_idx = INT32_MAX;
}
// Every lane offers one entry (cand false: none); the warp inserts those that belong.
__device__ __forceinline__ void top_offer(TopList& L, int top, int lane, bool cand, int key, int idx) {
    cand = cand && better(key, idx, L.kth_key, L.kth_idx);
    unsigned todo = __ballot_sync(0xffffffffu, cand);
    while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int k = __shfl_sync(0xffffffffu, key, src), i = __shfl_sync(0xffffffffu, idx, src);
        const int pk = __shfl_up_sync(0xffffffffu, L.key, 1), pi = __shfl_up_sync(0xffffffffu, L.idx, 1);
        const bool mine = better(L.key, L.idx, k, i);         // my entry stays ahead of the new one
        const bool prev = lane > 0 && !better(pk, pi, k, i);  // the one before me moves down to me
        if (!mine) {
            L.key = prev ? pk : k;
            L.idx = prev ? pi : i;
        }
        L.kth_key = __shfl_sync(0xffffffffu, L.key, top - 1);
        L.kth_idx = __shfl_sync(0xffffffffu, L.idx, top - 1);
        todo &= __ballot_sync(0xffffffffu, better(key, idx, L.kth_key, L.kth_idx));
    }
}

constexpr int FWD_THREADS = 256;
constexpr int FWD_WARPS = FWD_THREADS / 32;

// An entry of the alternatives as one number, larger first: the key, then the lower index.
// 0: none.
__device__ __forceinline__ uint64_t entry_of(int key, int idx) {
    return static_cast<uint64_t>(static_cast<uint32_t>(key) ^ 0x80000000u) << 32 | (0xffffffffu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ int entry_key(uint64_t e) { return static_cast<int>(static_cast<uint32_t>(e >> 32) ^ 0x80000000u); }
__device__ __forceinline__ int entry_index(uint64_t e) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)); }

// The k-th largest of the 32 lanes' keys, a lane's being the largest of its threads in all
// warps (KEY_NONE where fewer than k lanes have one).  Every warp finds it for itself.
__device__ __forceinline__ int kth_largest(const int* keys, int k, int lane) {
    int key = keys[lane];
#pragma unroll
    for (int w = 1; w < FWD_WARPS; ++w) key = max(key, keys[w * 32 + lane]);
    int place = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const int other = __shfl_sync(0xffffffffu, key, j);
        place += other > key || (other == key && j < lane) ? 1 : 0;
    }
    return __shfl_sync(0xffffffffu, key, __ffs(__ballot_sync(0xffffffffu, place == k - 1)) - 1);
}
constexpr int UNROLL = 4;  // 16-byte loads in flight per thread
constexpr int TURN = FWD_THREADS * UNROLL;  // vectors of a block's turn: each warp a run of 32 * UNROLL
constexpr int MAX_GROUPS = 16;  // groups of turns whose maxima a thread keeps
// Listed elements, and threads' groups to be read again.  A block has room at least for a run
// of so few vectors that fewer than k <= 32 lanes have one: 31 vectors, and the elements
// around them.
constexpr int TOP_LIST = 1024;

struct BlockResult {
    uint64_t best[LOGPROB_MAX_TOP];  // entries
    Stats st;
};

// A block's share of a row: whole vectors v0 to v1 of those from the row's first 16-byte
// boundary on, `head` elements in; and `nh` elements before and `nt` after all the vectors
// (fewer than a vector each, together a lane each of warp 0).
template <typename T>
struct Share {
    const T* x;
    int head, tail0, nh, nt, v0, v1;
    __device__ __forceinline__ const uint4* vectors() const { return reinterpret_cast<const uint4*>(x + head); }
    __device__ __forceinline__ int first(int tid) const { return v0 + (tid >> 5) * 32 * UNROLL + (tid & 31); }
    __device__ __forceinline__ int turns() const { return (v1 - v0 + TURN - 1) / TURN; }
    __device__ __forceinline__ int per_group() const { return (turns() + MAX_GROUPS - 1) / MAX_GROUPS; }
    __device__ __forceinline__ bool edge(int tid) const { return tid < nh + nt; }
    __device__ __forceinline__ int edge_index(int tid) const { return tid < nh ? tid : tail0 + tid - nh; }
};

// A maximum mx into the statistics: the first values, and then ever more rarely, raise m.
__device__ __forceinline__ void raise_max(Stats& st, float mx) {
    if (mx > st.m) {
        if (st.m != -INFINITY) {
            const float d = fmaxf((st.m - mx) * LOG2E, -200.f), c = ex2(d);
            st.q = c * (st.q + d * st.s);
            st.s *= c;
        }
        st.m = mx;
    }
}
// One value (-inf: none).
__device__ __forceinline__ void take_one(Stats& st, float v) {
    raise_max(st, v);
    const float y = max_nan((v - (st.m == -INFINITY ? 0.f : st.m)) * LOG2E, -200.f);
    const float e = ex2(y);
    st.s += e;
    st.q = fmaf(e, y, st.q);
}
// The first `cnt` of N vectors of values, none above st.m, none so far below it that the
// difference overflows.  The difference comes before the factor log2 e: a maximum of the type's
// lowest value (a row masked with it) times log2 e would overflow.
template <typename T, int N>
__device__ __forceinline__ void take(Stats& st, const uint4 (&raw)[N], int cnt) {
    constexpr int E = Elem<T>::VEC;
    const uint64_t nm = f2_make(-st.m, -st.m), l2e = f2_make(LOG2E, LOG2E);
    uint64_t s2 = 0, q2 = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (u >= cnt) break;
        uint64_t v[E / 2];
        Elem<T>::unpack_pairs(raw[u], v);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const uint64_t y = f2_mul(f2_add(v[i], nm), l2e);
            float y0, y1;
            f2_split(y, &y0, &y1);
            const uint64_t e = f2_make(ex2(y0), ex2(y1));
            s2 = f2_add(s2, e);
            q2 = f2_fma(e, y, q2);
        }
    }
    float s, q, sh, qh;
    f2_split(s2, &s, &sh);
    f2_split(q2, &q, &qh);
    st.s += s + sh;
    st.q += q + qh;
}

// Shared memory of the top k (none without them).
template <bool TOP>
struct TopShared {
    int group_max[MAX_GROUPS][FWD_THREADS];  // keys
    int thread_max[FWD_THREADS];
    uint64_t list[TOP_LIST];  // entries
    uint16_t again[TOP_LIST];  // groups to be read again: 256 * group + thread
    int count, agains;
};
template <>
struct TopShared<false> {};

// The statistics and the threads' maxima of a share whose values are not the common ones: in
// rows where nothing, or fewer than k values, are above what `not_below` makes of the masked
// ones, or where differences overflow.
template <typename T, bool TOP>
__device__ __noinline__ Stats exact_stats(const Share<T> sh, TopShared<TOP>& top, int tid) {
    constexpr int E = Elem<T>::VEC;
    Stats st = {-INFINITY, 0.f, 0.f};
    if (sh.edge(tid)) take_one(st, Elem<T>::load(sh.x[sh.edge_index(tid)]));
    int key_all = KEY_NONE, key_group = KEY_NONE, in_group = 0, group = 0;
#pragma unroll 1
    for (int base = sh.v0; base < sh.v1; base += TURN) {
        const int at = sh.first(tid) + (base - sh.v0);
        uint4 raw[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (at + u * 32 < sh.v1) raw[u] = sh.vectors()[at + u * 32];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (at + u * 32 >= sh.v1) break;
            float v[E], mx;
            Elem<T>::unpack(raw[u], v);
            mx = v[0];
#pragma unroll
            for (int i = 1; i < E; ++i) mx = fmaxf(mx, v[i]);
            raise_max(st, mx);
            const float m0 = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float y = max_nan((v[i] - m0) * LOG2E, -200.f), e = ex2(y);
                st.s += e;
                st.q = fmaf(e, y, st.q);
            }
            if (TOP) key_group = max(key_group, order_key(mx));
        }
        if constexpr (TOP) {
            key_all = max(key_all, key_group);
            if (++in_group == sh.per_group() || base + TURN >= sh.v1) {
                top.group_max[group++][tid] = key_group;
                key_group = KEY_NONE;
                in_group = 0;
            }
        }
    }
    if constexpr (TOP) top.thread_max[tid] = key_all;
    return st;
}

// Lists the share's elements that reach `least` (by the whole block; the list and `again` start
// empty).  Their number, or more than TOP_LIST where they may not all be listed.
template <typename T>
__device__ __forceinline__ int list_from(const Share<T>& sh, int least, TopShared<true>& top, int tid) {
    constexpr int E = Elem<T>::VEC;
    if (sh.edge(tid)) {
        const int i = sh.edge_index(tid), key = order_key(Elem<T>::load(sh.x[i]));
        if (key >= least) top.list[atomicAdd(&top.count, 1)] = entry_of(key, i);
    }
    const int per = sh.per_group();
    if (top.thread_max[tid] >= least) {
        for (int g = 0; g * per < sh.turns(); ++g) {
            if (top.group_max[g][tid] < least) continue;
            const int at = atomicAdd(&top.agains, 1);
            if (at < TOP_LIST) top.again[at] = static_cast<uint16_t>(g * FWD_THREADS + tid);
        }
    }
    __syncthreads();
    const int agains = top.agains, each = per * UNROLL;
    if (agains > TOP_LIST) return TOP_LIST + 1;
    for (int j = tid; j < agains * each; j += FWD_THREADS) {
        const int which_group = j / each, r = j - which_group * each;
        const int code = top.again[which_group];
        const int vec = sh.first(code % FWD_THREADS) + (code / FWD_THREADS * per + r / UNROLL) * TURN + r % UNROLL * 32;
        // (a list that is full already is not what the place is found by)
        if (vec >= sh.v1 || *static_cast<volatile int*>(&top.count) > TOP_LIST) continue;
        float v[E];
        Elem<T>::unpack(sh.vectors()[vec], v);
        unsigned which = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) which |= order_key(v[e]) >= least ? 1u << e : 0u;
        if (!which) continue;
        const int to = atomicAdd(&top.count, __popc(which));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = to + __popc(which & ((1u << e) - 1u));
            if ((which >> e & 1u) && i < TOP_LIST) top.list[i] = entry_of(order_key(v[e]), sh.head + vec * E + e);
        }
    }
    __syncthreads();
    return top.count;
}

// More elements reach the threshold `reach` than the list holds.  Many equal values (a masked
// row): the larger ones, and of the equal ones the first by index, up to k per warp and turn,
// until there are k.  Or the larger ones alone are too many: every warp walks its elements, its
// best k in order, and the lists become the entries.  The number of entries.
template <typename T>
__device__ __noinline__ int list_many(const Share<T> sh, int k, int reach, TopShared<true>& top, int tid) {
    constexpr int E = Elem<T>::VEC;
    const int lane = tid & 31;
    const uint4* xv = sh.vectors();
    __syncthreads();
    if (tid == 0) top.count = top.agains = 0;
    __syncthreads();
    const int larger = list_from(sh, reach + 1, top, tid);
    __syncthreads();
    if (larger + (FWD_WARPS + 2) * LOGPROB_MAX_TOP <= TOP_LIST) {
        if (sh.edge(tid)) {
            const int i = sh.edge_index(tid);
            if (order_key(Elem<T>::load(sh.x[i])) == reach) top.list[atomicAdd(&top.count, 1)] = entry_of(reach, i);
        }
        int equal = 0;  // listed by the turns
        for (int base = sh.v0; base < sh.v1 && equal < k; base += TURN) {
            int before = 0;  // equal values of the warp's earlier vectors
#pragma unroll 1
            for (int u = 0; u < UNROLL && before < k; ++u) {
                const int at = sh.first(tid) + (base - sh.v0) + u * 32;
                unsigned which = 0;
                if (at < sh.v1) {
                    float v[E];
                    Elem<T>::unpack(xv[at], v);
#pragma unroll
                    for (int e = 0; e < E; ++e) which |= order_key(v[e]) == reach ? 1u << e : 0u;
                }
                const int mine = __popc(which);
                int upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int left = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += left;
                }
                for (int place = before + upto - mine; which && place < k; which &= which - 1, ++place)
                    top.list[atomicAdd(&top.count, 1)] = entry_of(reach, sh.head + at * E + __ffs(which) - 1);
                before += __shfl_sync(0xffffffffu, upto, 31);
            }
            equal += __syncthreads_count(lane < min(before, k));
        }
        __syncthreads();
        return top.count;
    }
    TopList L;
    top_init(L);
    for (int base = sh.v0; base < sh.v1; base += TURN) {
        const int at = sh.first(tid) + (base - sh.v0);
        // indexes grow from turn to turn and from one row of vectors to the next: an equal
        // value never displaces, and what holds no larger one is passed over
#pragma unroll 1
        for (int u = 0; u < UNROLL; ++u) {
            const int vec = at + u * 32;
            float v[E];
            int most = KEY_NONE;
            if (vec < sh.v1) {
                Elem<T>::unpack(xv[vec], v);
#pragma unroll
                for (int e = 0; e < E; ++e) most = max(most, order_key(v[e]));
            }
            if (!__any_sync(0xffffffffu, most > L.kth_key)) continue;
#pragma unroll
            for (int e = 0; e < E; ++e)
                top_offer(L, k, lane, vec < sh.v1, vec < sh.v1 ? order_key(v[e]) : KEY_NONE, sh.head + vec * E + e);
        }
    }
    if (tid < 32) {
        const bool in = sh.edge(tid);
        const int i = sh.edge_index(tid);
        top_offer(L, k, lane, in, in ? order_key(Elem<T>::load(sh.x[i])) : KEY_NONE, i);
    }
    __syncthreads();
    if (tid == 0) top.count = 0;
    __syncthreads();
    if (lane < k && L.key != KEY_NONE) top.list[atomicAdd(&top.count, 1)] = entry_of(L.key, L.idx);
    __syncthreads();
    return top.count;
}

// The best `top` of n entries into their places: eight lanes count the entries ahead of one.
__device__ __forceinline__ void place_best(const uint64_t* list, int n, uint64_t* best, int top, int tid) {
    const int part = tid & 7;
    for (int j0 = 0; j0 < n; j0 += FWD_THREADS / 8) {
        const int j = j0 + tid / 8;
        const uint64_t mine = j < n ? list[j] : 0;
        int place = 0;
        for (int i = part; i < n; i += 8) place += list[i] > mine ? 1 : 0;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
        if (mine && part == 0 && place < top) best[place] = mine;
    }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(FWD_THREADS, 6) logprob_fwd_kernel(const LogprobParams p, int csize) {
    constexpr int E = Elem<T>::VEC;
    __shared__ Stats wst[FWD_WARPS];
    __shared__ BlockResult res;
    __shared__ TopShared<TOP> top;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / csize;
    const int rank = blockIdx.x % csize;
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;

    // The row from its first 16-byte boundary: `head` elements before it, then whole
    // vectors, then the tail.  Block `rank` of the cluster takes a run of vectors; the
    // first block also takes the head, the last one the tail.
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int head = min(mis ? E - mis : 0, p.vocab);
    const int nvec = (p.vocab - head) / E;
    const int per = (nvec + csize - 1) / csize;
    Share<T> sh;
    sh.x = x;
    sh.head = head;
    sh.tail0 = head + nvec * E;
    sh.v0 = min(rank * per, nvec);
    sh.v1 = min(sh.v0 + per, nvec);
    sh.nh = rank == 0 ? head : 0;
    sh.nt = rank == csize - 1 ? p.vocab - sh.tail0 : 0;

    pdl_wait_previous();  // (the next kernel starts after this one: its blocks, spread by what is free, would be uneven)
    // the target's logit, on its way from the start
    long long target = -1;
    float at_target = 0.f;
    if (p.logprob && tid == 0 && rank == 0) {
        target = p.target64 ? static_cast<const long long*>(p.targets)[row] : static_cast<const int*>(p.targets)[row];
        if (target >= 0 && target < p.vocab) at_target = Elem<T>::load(x[target]);
    }

    constexpr uint32_t LOW = Elem<T>::LOW;
    Stats st = {-INFINITY, 0.f, 0.f};
    if (sh.edge(tid)) take_one(st, Elem<T>::load(x[sh.edge_index(tid)]));
    const uint4* xv = sh.vectors();
    const int mine = sh.first(tid), per_group = sh.per_group();
    int key_all = KEY_NONE, key_group = KEY_NONE, in_group = 0, group = 0;
    for (int base = sh.v0; base < sh.v1; base += TURN) {
        const int at = mine + (base - sh.v0);
        uint4 raw[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) raw[u] = at + u * 32 < sh.v1 ? __ldcs(xv + at + u * 32) : make_uint4(LOW, LOW, LOW, LOW);
        uint32_t mw = LOW;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            raw[u].x = Elem<T>::not_below(raw[u].x);
            raw[u].y = Elem<T>::not_below(raw[u].y);
            raw[u].z = Elem<T>::not_below(raw[u].z);
            raw[u].w = Elem<T>::not_below(raw[u].w);
            mw = Elem<T>::max_word(mw, Elem<T>::max_word(Elem<T>::max_word(raw[u].x, raw[u].y), Elem<T>::max_word(raw[u].z, raw[u].w)));
        }
        const float mx = Elem<T>::word_max(mw);
        raise_max(st, mx);
        take<T, UNROLL>(st, raw, (sh.v1 - at + 31) / 32);  // vectors at + 32 u < v1
        if constexpr (TOP) {
            const int key = at < sh.v1 ? order_key(mx) : KEY_NONE;
            key_group = key > key_group ? key : key_group;
            key_all = key > key_all ? key : key_all;
            if (++in_group == per_group || base + TURN >= sh.v1) {
                top.group_max[group++][tid] = key_group;
                key_group = KEY_NONE;
                in_group = 0;
            }
        }
    }
    // the block's result: lanes, then warps, in a fixed order
    st = join<32>(st);
    if (lane == 0) wst[warp] = st;
    if constexpr (TOP) {
        top.thread_max[tid] = key_all;
        if (tid == 0) top.count = top.agains = 0;
        if (tid < LOGPROB_MAX_TOP) res.best[tid] = 0;
    }
    __syncthreads();
    st = join<FWD_WARPS>(wst[lane % FWD_WARPS]);
    int reach = KEY_NONE;
    if constexpr (TOP) reach = kth_largest(top.thread_max, p.top, lane);
    // Above these the values at LOW add nothing, exactly, and no difference overflows.
    constexpr float LEAST = sizeof(T) == 2 && LOW == Elem<__half>::LOW ? -65000.f : -9e29f;
    const bool common = st.m > LEAST && st.m < 1e38f && (!TOP || reach == KEY_NONE || key_value(reach) > LEAST);
    if (!common && sh.v0 < sh.v1) {
        __syncthreads();
        st = join<32>(exact_stats<T, TOP>(sh, top, tid));
        if (lane == 0) wst[warp] = st;
        __syncthreads();
        st = join<FWD_WARPS>(wst[lane % FWD_WARPS]);
        if constexpr (TOP) reach = kth_largest(top.thread_max, p.top, lane);
    }
    if constexpr (TOP) {
        int n = list_from(sh, reach, top, tid);
        if (n > TOP_LIST) n = list_many(sh, p.top, reach, top, tid);
        place_best(top.list, n, res.best, p.top, tid);
        __syncthreads();
    }
    if (csize > 1) {
        if (tid == 0) res.st = st;
        __syncwarp();
        cluster_sync();
        if (rank == 0) {
            if (warp == 0) {
                // eight lanes, four times over: the cluster's blocks (8 at most, a power of two)
                const uint32_t a = map_to_rank(&res.st, lane % csize);
                Stats b;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.m) : "r"(a) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.s) : "r"(a + 4) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.q) : "r"(a + 8) : "memory");
                if ((lane & 7) >= csize) b = {-INFINITY, 0.f, 0.f};
                st = join<8>(b);
            }
            if constexpr (TOP) {
                // the blocks' results are the entries: warp w takes those of block w
                if (warp < csize && lane < p.top) {
                    const uint32_t a = map_to_rank(&res.best[lane], warp);
                    uint64_t e;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(e) : "r"(a) : "memory");
                    top.list[warp * p.top + lane] = e;
                }
                __syncthreads();
                place_best(top.list, csize * p.top, res.best, p.top, tid);
                __syncthreads();
            }
        }
        __syncwarp();
        cluster_sync();  // no block leaves while its result may still be read
    }
    if (rank != 0 || warp != 0) return;
    const bool none = st.m == -INFINITY && st.s == 0.f;  // no logit above -inf (and no NaN)
    const float ls = logf(st.s);
    const float lse = none ? -INFINITY : st.m + ls;
    if (lane == 0) {
        if (p.lse) p.lse[row] = lse;
        if (p.entropy) p.entropy[row] = none ? 0.f : ls - LN2 * (st.q / st.s);
        if (p.logprob) {
            float lp = 0.f;  // a negative target: a position that does not count
            if (target >= p.vocab) lp = __int_as_float(0x7fc00000);  // no such token
            else if (target >= 0) lp = none ? -INFINITY : (at_target - st.m) - ls;
            p.logprob[row] = lp;
        }
    }
    if (TOP && lane < p.top) {
        const uint64_t e = res.best[lane];
        p.top_index[row * p.top + lane] = entry_index(e);
        p.top_logprob[row * p.top + lane] = none ? -INFINITY : (key_value(entry_key(e)) - st.m) - ls;
    }
}

constexpr int BWD_THREADS = 256;

// What every element of a row needs: u, v, lse, H, the target's column (or -1).
struct GradRow {
    float u, v, lse, h;
    int hit;
};

// Gradients of a vector of elements (the target's own term apart).
template <typename T, bool ENT>
__device__ __forceinline__ void grads_of(uint4 raw, float (&d)[Elem<T>::VEC], const GradRow& r) {
    constexpr int E = Elem<T>::VEC;
    const uint64_t nl = f2_make(-r.lse, -r.lse), l2e = f2_make(LOG2E, LOG2E), nu = f2_make(-r.u, -r.u);
    const uint64_t ln2 = f2_make(LN2, LN2), h = f2_make(r.h, r.h), nv = f2_make(-r.v, -r.v);
    uint64_t x[E / 2];
    Elem<T>::unpack_pairs(raw, x);
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const uint64_t y = f2_mul(f2_add(x[i], nl), l2e);
        float y0, y1;
        f2_split(y, &y0, &y1);
        const uint64_t pr = f2_make(ex2(y0), ex2(y1));
        // p (-v (log p + H) - u)
        const uint64_t g = f2_mul(pr, ENT ? f2_fma(nv, f2_fma(y, ln2, h), nu) : nu);
        f2_split(g, &d[2 * i], &d[2 * i + 1]);
        if (ENT) sum = f2_add(sum, g);
    }
    float a, b;
    f2_split(sum, &a, &b);
    if (ENT && a + b != a + b) {  // a masked logit: 0 times infinity
        float f[E];
        Elem<T>::unpack(raw, f);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float y = max_nan((f[i] - r.lse) * LOG2E, -200.f);
            d[i] = ex2(y) * fmaf(-r.v, fmaf(y, LN2, r.h), -r.u);
        }
    }
}
template <bool ENT>
__device__ __forceinline__ float grad_of(float x, int col, const GradRow& r) {
    const float y = max_nan((x - r.lse) * LOG2E, -200.f);
    float d = ENT ? ex2(y) * fmaf(-r.v, fmaf(y, LN2, r.h), -r.u) : -ex2(y) * r.u;
    if (col == r.hit) d += r.u;
    return d;
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(BWD_THREADS) logprob_bwd_kernel(const LogprobGradParams p, int segs) {
    constexpr int E = Elem<T>::VEC;
    const long long row = blockIdx.x / segs;
    const int seg = blockIdx.x % segs;
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    T* dx = static_cast<T*>(p.dlogits) + row * p.ldd;
    pdl_allow_next();
    pdl_wait_previous();
    GradRow r;
    r.lse = p.lse[row];
    const bool none = r.lse == -INFINITY;  // no distribution: the gradient is zero
    r.u = p.grad_logprob ? p.grad_logprob[row] : 0.f;
    r.v = ENT ? p.grad_entropy[row] : 0.f;
    r.h = ENT ? p.entropy[row] : 0.f;
    r.hit = -1;
    if (p.grad_logprob) {
        const long long t = p.target64 ? static_cast<const long long*>(p.targets)[row]
                                       : static_cast<const int*>(p.targets)[row];
        if (t < 0) r.u = 0.f;  // its log probability is the constant 0
        else if (t >= p.vocab) r.u = __int_as_float(0x7fc00000);
        else r.hit = static_cast<int>(t);
    }
    auto one = [&](int c) { dx[c] = Elem<T>::store(none ? 0.f : grad_of<ENT>(Elem<T>::load(x[c]), c, r)); };
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const bool vec = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
    if (vec) {
        const int head = min(mis ? E - mis : 0, p.vocab);
        const int nvec = (p.vocab - head) / E;
        const int tail0 = head + nvec * E;
        const int per = (nvec + segs - 1) / segs;
        const int v0 = min(seg * per, nvec), v1 = min(v0 + per, nvec);
        if (seg == 0 && threadIdx.x < head) one(threadIdx.x);
        if (seg == segs - 1 && threadIdx.x < p.vocab - tail0) one(tail0 + threadIdx.x);
        const uint4* xv = reinterpret_cast<const uint4*>(x + head);
        uint4* dv = reinterpret_cast<uint4*>(dx + head);
        const int hitv = r.hit >= head ? (r.hit - head) / E : -1;  // the vector of the target
        for (int base = v0 + threadIdx.x; base < v1; base += BWD_THREADS * UNROLL) {
            uint4 raw[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if (base + u * BWD_THREADS < v1) raw[u] = __ldcs(xv + base + u * BWD_THREADS);
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int i = base + u * BWD_THREADS;
                if (i < v1) {
                    float f[E];
                    if (none) {
#pragma unroll
                        for (int e = 0; e < E; ++e) f[e] = 0.f;
                    } else {
                        grads_of<T, ENT>(raw[u], f, r);
                        if (i == hitv) {
                            const int at = r.hit - head - i * E;
#pragma unroll
                            for (int e = 0; e < E; ++e)
                                if (e == at) f[e] += r.u;
                        }
                    }
                    __stcs(dv + i, Elem<T>::pack(f));
                }
            }
        }
    } else {
        // logits and gradient rows that sit differently to a 16-byte boundary: single elements
        const int per = (p.vocab + segs - 1) / segs;
        const int c1 = min((seg + 1) * per, p.vocab);
        for (int c = seg * per + threadIdx.x; c < c1; c += BWD_THREADS) one(c);
    }
}

template <typename T, bool TOP>
cudaError_t run_fwd(const LogprobParams& p, int csize, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows * csize));
    cfg.blockDim = dim3(FWD_THREADS);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logprob_fwd_kernel<T, TOP>, p, csize);
}

template <typename T>
cudaError_t run_bwd(const LogprobGradParams& p, int segs, cudaStream_t s) {
    const unsigned blocks = static_cast<unsigned>(p.rows * segs);
    return launch_pdl(p.grad_entropy ? logprob_bwd_kernel<T, true> : logprob_bwd_kernel<T, false>, dim3(blocks), dim3(BWD_THREADS), 0,
                      s, p, segs);
}

}  // namespace

cudaError_t launch_logprob_fwd(const LogprobParams& p, int sm_count, cudaStream_t s) {
    // blocks per row: more where the rows alone do not fill the SMs, as long as a block
    // still has half a turn of loads (8 KB)
    const long long bytes = static_cast<long long>(p.vocab) * dtype_size(p.dtype);
    int csize = 1;
    while (csize < 8 && p.rows * csize * 2 <= 2 * sm_count && bytes / (csize * 2) >= FWD_THREADS * UNROLL * 16 / 2) csize *= 2;
    switch (p.dtype) {
        case DT_F32: return p.top ? run_fwd<float, true>(p, csize, s) : run_fwd<float, false>(p, csize, s);
        case DT_BF16: return p.top ? run_fwd<__nv_bfloat16, true>(p, csize, s) : run_fwd<__nv_bfloat16, false>(p, csize, s);
        default: return p.top ? run_fwd<__half, true>(p, csize, s) : run_fwd<__half, false>(p, csize, s);
    }
}

int logprob_bwd_segments(int vocab, int dtype) {
    // whole turns of a block's loads (16 KB)
    const long long bytes = static_cast<long long>(vocab) * dtype_size(dtype);
    const long long turn = BWD_THREADS * UNROLL * 16;
    return static_cast<int>((bytes + turn - 1) / turn);
}

cudaError_t launch_logprob_bwd(const LogprobGradParams& p, cudaStream_t s) {
    const int segs = logprob_bwd_segments(p.vocab, p.dtype);
    switch (p.dtype) {
        case DT_F32: return run_bwd<float>(p, segs, s);
        case DT_BF16: return run_bwd<__nv_bfloat16>(p, segs, s);
        default: return run_bwd<__half>(p, segs, s);
    }
}

}  // namespace anvil
