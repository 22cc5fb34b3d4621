// router.hip -- hr_router_topk: the k largest logits of every token with their
// softmax weights, and hr_router_topk_grad, their gradient.
//
//   p = softmax(logits)          over the logits that are neither NaN nor -inf
//   ids, weights = the k largest logits and their p, by logit downward, equal
//                  logits (+0 and -0 are equal) by index upward
//   renormalised: weights = p / sum of the picked p
//
// Gradient of sum(dweights * weights), with c = sum_j dweights_j weights_j:
//
//   dlogits_e = p_e * (dweights of e's pick, or 0, - c)
//   renormalised: weights_j * (dweights_j - c) at the picks, 0 elsewhere
#include "rows.h"

#include <cfloat>
#include <type_traits>

namespace hr {

constexpr int kRouterThreads = 256;

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

struct RouterArgs {
    const void *logits;
    size_t stride;
    size_t tokens;
    float *weights;
    int32_t *ids;
    const float *dweights;   // the gradient only
    void *dlogits;
    size_t dstride;
    int experts;
    int k;
    int renormalize;
};

// Keys.  A logit and its index in one number, so that no two are equal and
// their order is "by logit downward, then by index upward": a 16-bit logit's
// order in the upper half of a word and the index's complement in the lower; a
// binary32 logit as binary64, the index in the bits that its fraction leaves
// free.  The smallest key stands for a logit that is never picked.
//
// Up to 8 picks of binary32 logits come from lists: every lane sorts its keys,
// and lists of the 8 largest are merged lane by lane.  Taking one pick after
// the other out of 256 binary32 logits costs about 100 instructions each, the
// lists 300 in all (32768 tokens, k=8: 15.1 against 11.4 us); out of 16-bit
// logits it costs 40 each, and lists were no faster (9.8 us either way).
template <int CTRL>
__device__ __forceinline__ double dpp_wide(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp<CTRL>(static_cast<uint32_t>(b)), hi = dpp<CTRL>(static_cast<uint32_t>(b >> 32));
    return __builtin_bit_cast(double, lo | hi << 32);
}

// The values of the lower and of the upper of two groups of D lanes (16 or
// 32), in the lanes of both.
template <int D>
__device__ __forceinline__ void both(double v, double &low, double &high) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t w[2] = {static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32)};
    uint64_t l = 0, h = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto r = D == 16 ? __builtin_amdgcn_permlane16_swap(w[i], w[i], false, false)
                               : __builtin_amdgcn_permlane32_swap(w[i], w[i], false, false);
        const uint32_t r0 = r[0], r1 = r[1];
        l |= static_cast<uint64_t>(r0) << (32 * i);
        h |= static_cast<uint64_t>(r1) << (32 * i);
    }
    low = __builtin_bit_cast(double, l);
    high = __builtin_bit_cast(double, h);
}

constexpr int kList = 8;

__device__ __forceinline__ void order2(double &a, double &b) {
    const double hi = __builtin_fmax(a, b);
    b = __builtin_fmin(a, b);
    a = hi;
}

// Eight keys downward: an odd-even merge network of 19 comparators.
__device__ __forceinline__ void sort8(double *k) {
    order2(k[0], k[1]); order2(k[2], k[3]); order2(k[4], k[5]); order2(k[6], k[7]);
    order2(k[0], k[2]); order2(k[1], k[3]); order2(k[4], k[6]); order2(k[5], k[7]);
    order2(k[1], k[2]); order2(k[5], k[6]);
    order2(k[0], k[4]); order2(k[1], k[5]); order2(k[2], k[6]); order2(k[3], k[7]);
    order2(k[2], k[4]); order2(k[3], k[5]);
    order2(k[1], k[2]); order2(k[3], k[4]); order2(k[5], k[6]);
}

// Eight keys that fall and rise, downward: 12 comparators.
__device__ __forceinline__ void sort_bitonic8(double (&k)[kList]) {
#pragma unroll
    for (int d = 4; d >= 1; d /= 2)
#pragma unroll
        for (int i = 0; i < kList; ++i)
            if ((i & d) == 0) order2(k[i], k[i + d]);
}

// The eight largest of two lists: the larger of one's i-th from the top and the
// other's i-th from the bottom.
template <int CTRL>
__device__ __forceinline__ void merge_lanes(double (&k)[kList]) {
    double m[kList];
#pragma unroll
    for (int i = 0; i < kList; ++i) m[i] = __builtin_fmax(k[i], dpp_wide<CTRL>(k[kList - 1 - i]));
#pragma unroll
    for (int i = 0; i < kList; ++i) k[i] = m[i];
    sort_bitonic8(k);
}

template <int D>
__device__ __forceinline__ void merge_groups(double (&k)[kList]) {
    double low[kList], high[kList];
#pragma unroll
    for (int i = 0; i < kList; ++i) both<D>(k[i], low[i], high[i]);
#pragma unroll
    for (int i = 0; i < kList; ++i) k[i] = __builtin_fmax(low[i], high[kList - 1 - i]);
    sort_bitonic8(k);
}

// The eight largest keys of L lanes with R each, downward, in every lane: each
// lane sorts its own, then lists are merged lane by lane.
template <int L, int R>
__device__ __forceinline__ void eight_largest(double (&key)[R], double (&list)[kList]) {
#pragma unroll
    for (int i = 0; i < R; i += kList) sort8(key + i);
#pragma unroll
    for (int i = 0; i < kList; ++i) list[i] = R == kList ? key[i] : __builtin_fmax(key[i], key[R - 1 - i]);
    if constexpr (R > kList) sort_bitonic8(list);
    merge_lanes<0xB1>(list);
    merge_lanes<0x4E>(list);
    merge_lanes<0x141>(list);
    if constexpr (L >= 16) merge_lanes<0x140>(list);
    if constexpr (L >= 32) merge_groups<16>(list);
    if constexpr (L >= 64) merge_groups<32>(list);
}

// The order of a binary32 logit as an unsigned number; 0 = never picked.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);      // -0 as +0
    const uint32_t u = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return x > -INFINITY ? u : 0u;
}

__device__ __forceinline__ float key_value(uint32_t u) {
    return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// R logits of lane t of L as they lie in memory (Raw), widened, and as keys:
// kVec consecutive ones (16 bytes) at a time, the lanes side by side, so that
// an access of the lanes covers whole lines.  (With a lane's R logits side by
// side the gradient of 32768 x 256 binary32 logits took 18.0 us against 11.4,
// of bfloat16 ones renormalised 6.4 against 5.2.)  What lies past the last
// logit reads as -infinity.
template <class T, int L>
__device__ __forceinline__ int logit_at(int r, int t) {
    return (r / T::kVec * L + t) * T::kVec + r % T::kVec;
}

struct Logits32 {
    static constexpr size_t kBytes = 4;
    static constexpr int kVec = 4;
    static constexpr bool kPacked = false;
    static __device__ __forceinline__ double key(float x, int e) {
        // a finite value beyond binary32 in infinity's place, which has no fraction
        const double d = x == INFINITY ? 0x1p200 : static_cast<double>(x + 0.0f);      // -0 as +0
        const uint64_t b = __builtin_bit_cast(uint64_t, d) | static_cast<uint32_t>(x >= 0.0f ? 0xFFFF - e : e);
        return x > -INFINITY ? __builtin_bit_cast(double, b) : -static_cast<double>(INFINITY);
    }
    static __device__ __forceinline__ bool picked(double key) { return key > -static_cast<double>(INFINITY); }
    static __device__ __forceinline__ float value(double key) {
        const uint64_t b = __builtin_bit_cast(uint64_t, key) & ~0xFFFFull;
        return static_cast<float>(__builtin_bit_cast(double, b));     // 2^200 becomes infinity again
    }
    static __device__ __forceinline__ int index(double key) {
        const int e = static_cast<int>(__builtin_bit_cast(uint64_t, key) & 0xFFFF);
        return key < 0.0 ? e : 0xFFFF - e;
    }
    template <int R>
    struct Raw {
        float x[R];
    };
    template <int L, int R>
    static __device__ __forceinline__ void load(const void *row, int t, int n, Raw<R> &raw) {
        const float *p = static_cast<const float *>(row);
#pragma unroll
        for (int q = 0; q < R / 4; ++q) {
            const int e = logit_at<Logits32, L>(4 * q, t);
            if (e + 4 <= n) {
                const f32x4 v = *reinterpret_cast<const f32x4_row *>(p + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) raw.x[4 * q + i] = v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) raw.x[4 * q + i] = e + i < n ? p[e + i] : -INFINITY;
            }
        }
    }
    template <int R>
    static __device__ __forceinline__ void widen(const Raw<R> &raw, float (&x)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = raw.x[r];
    }
    static __device__ __forceinline__ float narrow1(float v) { return v; }
    static __device__ __forceinline__ u32x4 narrow(const float *x) {
        return __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]});
    }
    // The last unit of a row of n, whose value e is the unit's first.
    static __device__ __forceinline__ void store_part(void *row, int e, int n, u32x4 v) {
        uint32_t *p = static_cast<uint32_t *>(row) + e;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (e + i < n) p[i] = v[i];
    }
};

template <class E>
struct Logits16 {
    static constexpr size_t kBytes = 2;
    static constexpr int kVec = 8;
    static constexpr bool kPacked = true;
    static constexpr uint32_t kInf = std::is_same<E, F16>::value ? 0x7C00u : 0x7F80u;
    static constexpr uint32_t kNone = (0x8000u | kInf) * 0x10001u;
    template <int R>
    struct Raw {
        uint32_t w[R / 2];           // two logits to a word
    };
    template <int L, int R>
    static __device__ __forceinline__ void load(const void *row, int t, int n, Raw<R> &raw) {
        const uint16_t *p = static_cast<const uint16_t *>(row);
#pragma unroll
        for (int q = 0; q < R / 8; ++q) {
            const int e = logit_at<Logits16, L>(8 * q, t);
            if (e + 8 <= n) {
                const u32x4 v = load_vec<false>(p + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) raw.w[4 * q + i] = v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint32_t lo = e + i < n ? p[e + i] : kNone & 0xFFFFu;
                    const uint32_t hi = e + i + 1 < n ? p[e + i + 1] : kNone >> 16;
                    raw.w[4 * q + i / 2] = lo | hi << 16;
                }
            }
        }
    }
    template <int R>
    static __device__ __forceinline__ void widen(const Raw<R> &raw, float (&x)[R]) {
#pragma unroll
        for (int q = 0; q < R / 8; ++q) {
            float f[8];
            Wide<E>::widen(u32x4{raw.w[4 * q], raw.w[4 * q + 1], raw.w[4 * q + 2], raw.w[4 * q + 3]}, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[8 * q + i] = f[i];
        }
    }
    static __device__ __forceinline__ uint16_t narrow1(float v) { return Wide<E>::narrow1(v); }
    static __device__ __forceinline__ u32x4 narrow(const float *x) {
        const float f[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
        return Wide<E>::narrow(f);
    }
    static __device__ __forceinline__ void store_part(void *row, int e, int n, u32x4 v) {
        uint16_t *p = static_cast<uint16_t *>(row) + e;
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (e + i < n) p[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1)));
    }
    // Two logits to their orders, 1 and up; 0 = never picked.  A negative w is
    // at 2^16 - w, others at 2^15 + w, so that both zeros meet in 2^15, with
    // kNaN NaNs above +infinity and kNaN + 1 numbers up to -infinity.  Adding
    // kNaN takes the upper NaNs round past zero, and a subtraction that stops
    // at zero takes all of these away.
    static constexpr uint16_t kNaN = 0x7FFF - kInf;
    static __device__ __forceinline__ uint32_t orders(uint32_t w) {
        const i16x2 v = __builtin_bit_cast(i16x2, w), sign = v >> 15;
        const u16x2 flip = __builtin_bit_cast(u16x2, w ^ (__builtin_bit_cast(uint32_t, sign) | 0x80008000u));
        const u16x2 u = flip - __builtin_bit_cast(u16x2, sign) + u16x2{kNaN, kNaN};
        constexpr uint16_t kDrop = 2 * kNaN + 1;
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(u, u16x2{kDrop, kDrop}));
    }
    // Keys without the lane's part of the index: key(r, t) = k[r] - lane_key(t).
    template <int L, int R>
    static __device__ __forceinline__ void keys(const Raw<R> &raw, uint32_t (&k)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t o = orders(raw.w[r / 2]);
            k[r] = (r & 1 ? o & 0xFFFF0000u : o << 16) + (0xFFFFu - logit_at<Logits16, L>(r, 0));
        }
    }
    static __device__ __forceinline__ uint32_t lane_key(int t) { return kVec * t; }
    static __device__ __forceinline__ bool picked(uint32_t key) { return key > 0xFFFFu; }
    static __device__ __forceinline__ int index(uint32_t key) { return static_cast<int>(0xFFFFu - (key & 0xFFFFu)); }
    static __device__ __forceinline__ float value(uint32_t key) {
        const uint32_t u = (key >> 16) + kNaN + 1;
        return Wide<E>::widen1(static_cast<uint16_t>(u >= 0x8000u ? u ^ 0x8000u : 0x10000u - u));
    }
};

// exp(x - top) of R logits and their sum: 0 for -infinity and NaN, and for
// everything where top is -infinity (nothing to pick); where top is +infinity,
// 1 for each +infinity.  The instruction gives 2^p for p = (x - top) log2(e)
// rounded to 24 bits, which alone is up to |p| 2^-25 of the result; what the
// rounding left out, times ln 2, is (x - top) - p ln 2, and corrects it.  So a
// term is off by the instruction's last place and a rounding, whatever its size.
// (32768 x 256 bfloat16 logits, k=8, forward and back: 8.4 and 7.6 us uncorrected,
// 8.7 and 8.0 so.)
// Infinities and NaN come out as NaN, which the clamp to 0..1, a modifier of the
// last operation, makes 0.
template <int R>
__device__ __forceinline__ float exp_all(float (&x)[R], float top) {
    constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
    const float from = top == -INFINITY ? 0.0f : top;
    float y[R], total = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float d = x[r] - from, p = d * kLog2e, e = __builtin_amdgcn_exp2f(p);
        y[r] = __builtin_amdgcn_fmed3f(fmaf(e, fmaf(-p, kLn2, d), e), 0.0f, 1.0f);
        total += y[r];
    }
    if (__ballot(top == INFINITY) != 0) {
        total = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            y[r] = top != INFINITY ? y[r] : x[r] == INFINITY ? 1.0f : 0.0f;
            total += y[r];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = y[r];
    return total;
}

// LIST: up to 8 picks of binary32 logits.  32768 tokens of 256, k=8, in a graph:
// bfloat16 8.7 us, 7.4 renormalised, where the logits' way from memory takes 3;
// binary32 11.1 and 10.4.  Bound by instructions, about 510 a wave of four
// bfloat16 tokens: keys 85 (made one by one they were 190, and took 0.3 to 0.8 us
// more), picks 37 each, exponentials 96 and half as much again for their quarter
// rate.
template <class T, int L, int R, bool LIST>
__global__ __launch_bounds__(kRouterThreads) void router_topk(RouterArgs a) {
    constexpr int kTokens = kRouterThreads / L;
    const int t = threadIdx.x % L;
    const size_t token = static_cast<size_t>(blockIdx.x) * kTokens + threadIdx.x / L;
    const bool there = token < a.tokens;
    typename T::template Raw<R> raw;
    T::template load<L>(static_cast<const char *>(a.logits) + (there ? token : 0) * a.stride * T::kBytes, t,
                        there ? a.experts : 0, raw);

    // the picks, lane j keeping pick j, and the largest logit
    float top = -INFINITY, v = 0.0f;
    int id = -1;
    if constexpr (T::kPacked) {
        // The next pick is the largest key below the last one, that is the
        // largest difference to it modulo 2^32: nothing has to be taken out.
        // (Keys of what is never picked differ too, and there are k keys at least.)
        uint32_t key[R];
        T::template keys<L>(raw, key);
        uint32_t m = key[0];
#pragma unroll
        for (int r = 1; r < R; ++r) m = m > key[r] ? m : key[r];
        const uint32_t first = max_lanes<L>(m - T::lane_key(t));
        uint32_t last = first, mine = t == 0 ? first : 0;
        for (int j = 1; j < a.k; ++j) {
            const uint32_t base = last + T::lane_key(t);
            m = key[0] - base;
#pragma unroll
            for (int r = 1; r < R; ++r) {
                const uint32_t d = key[r] - base;
                m = m > d ? m : d;
            }
            last += max_lanes<L>(m);
            mine = t == j ? last : mine;
        }
        if (T::picked(first)) top = T::value(first);
        if (T::picked(mine)) {
            v = T::value(mine);
            id = T::index(mine);
        }
    } else if constexpr (LIST) {
        double key[R], list[kList];
#pragma unroll
        for (int r = 0; r < R; ++r) key[r] = T::key(raw.x[r], logit_at<T, L>(r, t));
        eight_largest<L>(key, list);
        double mine = list[0];
#pragma unroll
        for (int i = 1; i < kList; ++i) mine = t == i ? list[i] : mine;
        if (T::picked(list[0])) top = T::value(list[0]);
        if (t < a.k && T::picked(mine)) {
            v = T::value(mine);
            id = T::index(mine);
        }
    } else {
        uint32_t key[R];
#pragma unroll
        for (int r = 0; r < R; ++r) key[r] = order_key(raw.x[r]);
        uint32_t best = 0, mine = 0;
        for (int j = 0; j < a.k; ++j) {
            uint32_t m = key[0];
#pragma unroll
            for (int r = 1; r < R; ++r) m = m > key[r] ? m : key[r];
            m = max_lanes<L>(m);
            // the lowest index with that key: as the largest complement
            uint32_t at = 0;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) at = key[r] == m ? ~static_cast<uint32_t>(logit_at<T, L>(r, t)) : at;
            const int e = static_cast<int>(~max_lanes<L>(at));
#pragma unroll
            for (int r = 0; r < R; ++r) key[r] = logit_at<T, L>(r, t) == e ? 0u : key[r];
            best = j == 0 ? m : best;
            mine = t == j ? m : mine;
            id = t == j && m != 0 ? e : id;
        }
        if (best != 0) top = key_value(best);
        v = key_value(mine);
    }

    float w[1] = {id >= 0 ? v : -INFINITY};
    float total = exp_all(w, top);
    if (!a.renormalize) {
        float x[R];
        T::widen(raw, x);
        total = exp_all(x, top);
    }
    total = sum_lanes<L>(total);
    if (there && t < a.k) {
        a.weights[token * a.k + t] = id >= 0 ? w[0] / total : 0.0f;
        a.ids[token * a.k + t] = id;
    }
}

// A wave's accesses of LDS are carried out in order, so between lanes of one
// wave it is only the compiler that has to keep it.
__device__ __forceinline__ void order_lds() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// p * (0 - c) for every logit, put together in LDS, where the picks' own
// weights * (dweights - c) take their places; a token's lanes are in one wave.
// 32768 tokens of 256, k=8, in a graph: bfloat16 8.0 us, binary32 11.6 (67 MB, 5.8
// TB/s from the last-level cache), renormalised 5.4 and 7.8.
template <class T, int L, int R>
__global__ __launch_bounds__(kRouterThreads) void router_topk_grad(RouterArgs a) {
    constexpr int kTokens = kRouterThreads / L, kUnits = R / T::kVec;
    // by units of a lane's logits, the lanes side by side: no two lanes of an
    // access share a bank (with a lane's logits side by side, four did)
    __shared__ u32x4 out[kTokens][kUnits][L];
    const int t = threadIdx.x % L;
    const int slot = threadIdx.x / L;
    const size_t token = static_cast<size_t>(blockIdx.x) * kTokens + slot;
    const bool there = token < a.tokens;
    typename T::template Raw<R> raw;
    if (!a.renormalize)
        T::template load<L>(static_cast<const char *>(a.logits) + (there ? token : 0) * a.stride * T::kBytes, t,
                            there ? a.experts : 0, raw);
    int id = -1;
    float g = 0.0f, w = 0.0f;
    if (there && t < a.k) {
        id = a.ids[token * a.k + t];
        if (id >= 0 && id < a.experts) {
            g = a.dweights[token * a.k + t];
            w = a.weights[token * a.k + t];
        } else {
            id = -1;
        }
    }
    const float c = sum_lanes<L>(id >= 0 ? g * w : 0.0f);
    if (a.renormalize) {
#pragma unroll
        for (int q = 0; q < kUnits; ++q) out[slot][q][t] = u32x4{0, 0, 0, 0};
    } else {
        float x[R];
        T::widen(raw, x);
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r) top = fmaxf(top, x[r]);     // a NaN is no maximum
        top = reduce_lanes<L>(top, [](float p, float q) { return fmaxf(p, q); });
        const float total = sum_lanes<L>(exp_all(x, top));
        const float scale = total > 0.0f ? -c / total : -c;
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] *= scale;
#pragma unroll
        for (int q = 0; q < kUnits; ++q) out[slot][q][t] = T::narrow(x + q * T::kVec);
    }
    order_lds();
    if (id >= 0) {
        const auto v = T::narrow1(w * (g - c));
        char *unit = reinterpret_cast<char *>(&out[slot][id / (T::kVec * L)][id / T::kVec % L]);
        __builtin_memcpy(unit + id % T::kVec * sizeof(v), &v, sizeof(v));
    }
    order_lds();
    if (!there) return;
    char *row = static_cast<char *>(a.dlogits) + token * a.dstride * T::kBytes;
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        const int e = logit_at<T, L>(q * T::kVec, t);
        const u32x4 v = out[slot][q][t];
        if (e + T::kVec <= a.experts)
            store_vec<false>(v, row + e * T::kBytes);
        else
            T::store_part(row, e, a.experts, v);
    }
}

namespace {

template <class T, int L, int R>
hipError_t launch_router(const RouterArgs &a, bool grad, hipStream_t s) {
    constexpr int kTokens = kRouterThreads / L;
    const unsigned grid = static_cast<unsigned>((a.tokens + kTokens - 1) / kTokens);
    if (grad)
        hipLaunchKernelGGL((router_topk_grad<T, L, R>), dim3(grid), dim3(kRouterThreads), 0, s, a);
    else if constexpr (T::kPacked)
        hipLaunchKernelGGL((router_topk<T, L, R, false>), dim3(grid), dim3(kRouterThreads), 0, s, a);
    else if (L == 8 || a.k <= kList)
        hipLaunchKernelGGL((router_topk<T, L, R, true>), dim3(grid), dim3(kRouterThreads), 0, s, a);
    else if constexpr (L > 8)
        hipLaunchKernelGGL((router_topk<T, L, R, false>), dim3(grid), dim3(kRouterThreads), 0, s, a);
    return hipGetLastError();
}

// Lanes per token: enough for one pick each and for the logits at 8 or 16 per
// lane.
template <class T>
hipError_t launch_router(const RouterArgs &a, bool grad, hipStream_t s) {
    if (a.experts <= 64 && a.k <= 8) return launch_router<T, 8, 8>(a, grad, s);
    if (a.experts <= 128 && a.k <= 16) return launch_router<T, 16, 8>(a, grad, s);
    if (a.experts <= 256 && a.k <= 16) return launch_router<T, 16, 16>(a, grad, s);
    if (a.experts <= 256) return launch_router<T, 32, 8>(a, grad, s);
    if (a.experts <= 512) return launch_router<T, 32, 16>(a, grad, s);
    return launch_router<T, 64, 16>(a, grad, s);
}

hr_status router_impl(RouterArgs &a, hr_dtype dtype, bool grad, hr_stream_t stream) {
    if (a.experts < 1 || a.k < 1 || a.k > a.experts) return HR_ERR_INVALID_ARG;
    if (dtype != HR_DTYPE_F16 && dtype != HR_DTYPE_BF16 && dtype != HR_DTYPE_F32) return HR_ERR_INVALID_ARG;
    if (a.experts > HR_ROUTER_MAX_EXPERTS || a.k > HR_ROUTER_MAX_K || a.tokens > HR_ROUTER_MAX_TOKENS) return HR_ERR_TOO_LARGE;
    if (a.tokens == 0) return HR_OK;
    const bool reads = !grad || !a.renormalize;
    if (a.weights == nullptr || a.ids == nullptr || (reads && a.logits == nullptr)) return HR_ERR_INVALID_ARG;
    if (grad && (a.dweights == nullptr || a.dlogits == nullptr)) return HR_ERR_INVALID_ARG;
    const size_t size = dtype == HR_DTYPE_F32 ? 4 : 2, E = static_cast<size_t>(a.experts);
    if (!row_stride(a.tokens, E, &a.stride, size) || !row_stride(a.tokens, E, &a.dstride, size))
        return HR_ERR_INVALID_ARG;
    if (!aligned(a.logits, size) || !aligned(a.dlogits, size) || !aligned(a.weights, 4) || !aligned(a.ids, 4) ||
        !aligned(a.dweights, 4))
        return HR_ERR_ALIGNMENT;
    const Region logits = {reads ? a.logits : nullptr, a.tokens, E * size, a.stride * size};
    const Region dlogits = {a.dlogits, a.tokens, E * size, a.dstride * size};
    const size_t per = static_cast<size_t>(a.k) * 4;
    const Region weights = {a.weights, a.tokens, per, per}, ids = {a.ids, a.tokens, per, per};
    const Region dweights = {a.dweights, a.tokens, per, per};
    if (grad) {
        if (regions_overlap(dlogits, weights) || regions_overlap(dlogits, ids) || regions_overlap(dlogits, dweights) ||
            (regions_overlap(dlogits, logits) && !regions_same(dlogits, logits)))
            return HR_ERR_INVALID_ARG;
    } else if (regions_overlap(weights, ids) || regions_overlap(weights, logits) || regions_overlap(ids, logits)) {
        return HR_ERR_INVALID_ARG;
    }
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = dtype == HR_DTYPE_F32   ? launch_router<Logits32>(a, grad, s)
                         : dtype == HR_DTYPE_F16 ? launch_router<Logits16<F16>>(a, grad, s)
                                                 : launch_router<Logits16<BF16>>(a, grad, s);
    return e == hipSuccess ? HR_OK : HR_ERR_HIP;
}

}  // namespace

}  // namespace hr

using namespace hr;

extern "C" HR_API hr_status hr_router_topk(const void *logits, hr_dtype dtype, size_t tokens, int experts,
                                           size_t logits_stride, int k, int renormalize, float *weights, int32_t *ids,
                                           hr_stream_t stream) {
    RouterArgs a{};
    a.logits = logits;
    a.stride = logits_stride;
    a.tokens = tokens;
    a.weights = weights;
    a.ids = ids;
    a.experts = experts;
    a.k = k;
    a.renormalize = renormalize != 0;
    return router_impl(a, dtype, false, stream);
}

extern "C" HR_API hr_status hr_router_topk_grad(const float *dweights, const float *weights, const int32_t *ids,
                                                const void *logits, hr_dtype dtype, size_t tokens, int experts,
                                                size_t logits_stride, int k, int renormalize, void *dlogits,
                                                size_t dlogits_stride, hr_stream_t stream) {
    RouterArgs a{};
    a.logits = logits;
    a.stride = logits_stride;
    a.tokens = tokens;
    a.weights = const_cast<float *>(weights);
    a.ids = const_cast<int32_t *>(ids);
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.dstride = dlogits_stride;
    a.experts = experts;
    a.k = k;
    a.renormalize = renormalize != 0;
    return router_impl(a, dtype, true, stream);
}
