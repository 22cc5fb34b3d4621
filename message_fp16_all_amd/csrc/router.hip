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

// exp(d) for d <= 0, to about two units in the last place: d * log2(e) as a
// rounded product and its remainder, 2^x of the first by the hardware, the
// second to first order.  Below -200 the result is 0 in binary32 all the same.
__device__ __forceinline__ float exp_down(float d) {
    constexpr float kLog2e = 1.44269504088896341f;              // rounded to binary32
    constexpr float kLog2eLow = 1.92596299112661746e-8f;        // log2(e) - kLog2e
    constexpr float kLn2 = 0.693147180559945309f;
    d = fmaxf(d, -200.0f);
    const float a = d * kLog2e;
    const float r = fmaf(d, kLog2e, -a) + d * kLog2eLow;
    const float p = __builtin_amdgcn_exp2f(a);
    return fmaf(p, r * kLn2, p);
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

// R consecutive logits of one lane as they lie in memory (Raw), widened, and
// as keys.  What lies past the last logit reads as -infinity.
struct Logits32 {
    static constexpr size_t kBytes = 4;
    static constexpr bool kPacked = false;
    template <int R>
    struct Raw {
        float x[R];
    };
    template <int R>
    static __device__ __forceinline__ void load(const void *row, int e0, int n, Raw<R> &raw) {
        const float *p = static_cast<const float *>(row) + e0;
        if (e0 + R <= n) {
#pragma unroll
            for (int q = 0; q < R / 4; ++q) {
                const f32x4 v = *reinterpret_cast<const f32x4_row *>(p + 4 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) raw.x[4 * q + i] = v[i];
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) raw.x[r] = e0 + r < n ? p[r] : -INFINITY;
        }
    }
    template <int R>
    static __device__ __forceinline__ void widen(const Raw<R> &raw, float (&x)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = raw.x[r];
    }
    template <int R>
    static __device__ __forceinline__ void store(void *row, int e0, int n, const float (&x)[R]) {
        float *p = static_cast<float *>(row) + e0;
        if (e0 + R <= n) {
#pragma unroll
            for (int q = 0; q < R / 4; ++q)
                *reinterpret_cast<f32x4_row *>(p + 4 * q) = f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (e0 + r < n) p[r] = x[r];
        }
    }
};

template <class E>
struct Logits16 {
    static constexpr size_t kBytes = 2;
    static constexpr bool kPacked = true;
    static constexpr uint32_t kInf = std::is_same<E, F16>::value ? 0x7C00u : 0x7F80u;
    static constexpr uint32_t kNone = (0x8000u | kInf) * 0x10001u;
    template <int R>
    struct Raw {
        uint32_t w[R / 2];           // two logits to a word
    };
    template <int R>
    static __device__ __forceinline__ void load(const void *row, int e0, int n, Raw<R> &raw) {
        const uint16_t *p = static_cast<const uint16_t *>(row) + e0;
        if (e0 + R <= n) {
#pragma unroll
            for (int q = 0; q < R / 8; ++q) {
                const u32x4 v = load_vec<false>(p + 8 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) raw.w[4 * q + i] = v[i];
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; r += 2) {
                const uint32_t lo = e0 + r < n ? p[r] : kNone & 0xFFFFu, hi = e0 + r + 1 < n ? p[r + 1] : kNone >> 16;
                raw.w[r / 2] = lo | hi << 16;
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
    template <int R>
    static __device__ __forceinline__ void store(void *row, int e0, int n, const float (&x)[R]) {
#pragma unroll
        for (int q = 0; q < R / 8; ++q) {
            const int e = e0 + 8 * q;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = x[8 * q + i];
            const u32x4 v = Wide<E>::narrow(f);
            uint16_t *p = static_cast<uint16_t *>(row) + e;
            if (e + 8 <= n) {
                store_vec<false>(v, p);
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (e + i < n) p[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1)));
            }
        }
    }
    // A logit's order in the upper half of a word and its index's complement in
    // the lower, so that no two are equal; 0 = never picked.  `bits` holds the
    // logit in its upper half and zeros below.
    static __device__ __forceinline__ uint32_t key(uint32_t bits, int e) {
        bits = bits == 0x80000000u ? 0u : bits;                 // -0 as +0
        const uint32_t u = bits ^ (static_cast<uint32_t>(static_cast<int32_t>(bits) >> 31) | 0x80000000u);
        // above -infinity (whose order is 0x7FFF - kInf) and up to +infinity
        constexpr uint32_t kLow = (0x8000u - kInf) << 16, kHigh = (0x8000u | kInf) << 16 | 0xFFFFu;
        return u - kLow <= kHigh - kLow ? (u & 0xFFFF0000u) | (0xFFFFu - e) : 0u;
    }
    template <int R>
    static __device__ __forceinline__ void keys(const Raw<R> &raw, int e0, uint32_t (&k)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) k[r] = key(r & 1 ? raw.w[r / 2] & 0xFFFF0000u : raw.w[r / 2] << 16, e0 + r);
    }
    static __device__ __forceinline__ float value(uint32_t key) {
        const uint32_t u = key >> 16;
        return Wide<E>::widen1(static_cast<uint16_t>(u & 0x8000u ? u ^ 0x8000u : ~u));
    }
};

// exp(x - top) of R logits and their sum: 0 for -infinity and NaN, and for
// everything where top is -infinity (nothing to pick); where top is +infinity,
// 1 for each +infinity.
template <int R>
__device__ __forceinline__ float exp_all(float (&x)[R], float top) {
    if (top == INFINITY) {
        // the largest number in infinity's place: its difference to itself is 0
        top = FLT_MAX;
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = x[r] == INFINITY ? FLT_MAX : -INFINITY;
    }
    float total = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        // (a difference that is NaN or -infinity ends as an exponent that gives 0)
        x[r] = exp_down(x[r] - top);
        total += x[r];
    }
    return total;
}

// One token per L lanes; lane t holds the R logits t * R, t * R + 1, ..
template <class T, int L, int R>
__global__ __launch_bounds__(kRouterThreads) void router_topk(RouterArgs a) {
    constexpr int kTokens = kRouterThreads / L;
    const int t = threadIdx.x % L;
    const size_t token = static_cast<size_t>(blockIdx.x) * kTokens + threadIdx.x / L;
    const bool there = token < a.tokens;
    const int e0 = t * R;
    typename T::template Raw<R> raw;
    T::load(static_cast<const char *>(a.logits) + (there ? token : 0) * a.stride * T::kBytes, e0,
            there ? a.experts : 0, raw);

    // the picks, lane j keeping pick j, and the largest logit
    float top = 0.0f, v = 0.0f;
    int id = -1;
    if constexpr (T::kPacked) {
        // The next pick is the largest key below the last one, that is the
        // largest difference to it modulo 2^32: nothing has to be taken out.
        uint32_t key[R];
        T::keys(raw, e0, key);
        uint32_t last = 0, first = 0, mine = 0;
        for (int j = 0; j < a.k; ++j) {
            uint32_t m = key[0] - last;
#pragma unroll
            for (int r = 1; r < R; ++r) {
                const uint32_t d = key[r] - last;
                m = m > d ? m : d;
            }
            m = max_lanes<L>(m) + last;
            last = j > 0 && last == 0 ? 0u : m;                 // nothing was left
            first = j == 0 ? last : first;
            mine = t == j ? last : mine;
        }
        top = first != 0 ? T::value(first) : -INFINITY;
        if (mine != 0) {
            v = T::value(mine);
            id = static_cast<int>(0xFFFFu - (mine & 0xFFFFu));
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
            for (int r = R - 1; r >= 0; --r) at = key[r] == m ? ~static_cast<uint32_t>(e0 + r) : at;
            const int e = static_cast<int>(~max_lanes<L>(at));
#pragma unroll
            for (int r = 0; r < R; ++r) key[r] = e0 + r == e ? 0u : key[r];
            best = j == 0 ? m : best;
            mine = t == j ? m : mine;
            id = t == j && m != 0 ? e : id;
        }
        top = best != 0 ? key_value(best) : -INFINITY;
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

template <class T, int L, int R>
__global__ __launch_bounds__(kRouterThreads) void router_topk_grad(RouterArgs a) {
    constexpr int kTokens = kRouterThreads / L;
    __shared__ float picked[kTokens][L * R];
    const int t = threadIdx.x % L;
    const int slot = threadIdx.x / L;
    const size_t token = static_cast<size_t>(blockIdx.x) * kTokens + slot;
    const bool there = token < a.tokens;
    const int e0 = t * R;
    typename T::template Raw<R> raw;
    if (!a.renormalize)
        T::load(static_cast<const char *>(a.logits) + (there ? token : 0) * a.stride * T::kBytes, e0,
                there ? a.experts : 0, raw);
#pragma unroll
    for (int r = 0; r < R; ++r) picked[slot][e0 + r] = 0.0f;
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
    __syncthreads();
    if (id >= 0) picked[slot][id] = a.renormalize ? w * (g - c) : g;
    __syncthreads();

    float x[R];
    if (a.renormalize) {
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = picked[slot][e0 + r];
    } else {
        T::widen(raw, x);
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r) top = fmaxf(top, x[r]);     // a NaN is no maximum
        top = reduce_lanes<L>(top, [](float p, float q) { return fmaxf(p, q); });
        const float total = sum_lanes<L>(exp_all(x, top));
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = x[r] * inv * (picked[slot][e0 + r] - c);
    }
    if (there && e0 < a.experts)
        T::store(static_cast<char *>(a.dlogits) + token * a.dstride * T::kBytes, e0, a.experts, x);
}

namespace {

template <class T, int L, int R>
hipError_t launch_router(const RouterArgs &a, bool grad, hipStream_t s) {
    constexpr int kTokens = kRouterThreads / L;
    const unsigned grid = static_cast<unsigned>((a.tokens + kTokens - 1) / kTokens);
    if (grad)
        hipLaunchKernelGGL((router_topk_grad<T, L, R>), dim3(grid), dim3(kRouterThreads), 0, s, a);
    else
        hipLaunchKernelGGL((router_topk<T, L, R>), dim3(grid), dim3(kRouterThreads), 0, s, a);
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
