// rows.h -- helpers of the kernels that work on rows of 16-bit values (norms,
// expert rows, router logits); not exported.
//
// A row is read and written in units of 8 values (16 bytes).  Rows may start
// at any address of a value: gfx950 serves unaligned 16-byte global accesses,
// so the unit type promises no alignment, and the same instruction carries
// aligned and unaligned rows.  (Rows at a multiple of 4 bytes run at full speed;
// at odd 2-byte addresses a norm of 4999 x 5120 took 48 us against 39.)
#pragma once

#include "hr_internal.h"

namespace hr {

typedef u32x4 u32x4_byte __attribute__((aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_row __attribute__((aligned(1)));
typedef uint32_t u32_row __attribute__((aligned(1)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_row __attribute__((aligned(4)));

constexpr int kWave = 64;

// The 8 values of a unit, widened exactly to binary32, and narrowed back with
// one rounding to nearest even each.
template <class E>
struct Wide;

template <>
struct Wide<F16> {
    static __device__ __forceinline__ float widen1(uint16_t v) {
        return static_cast<float>(__builtin_bit_cast(_Float16, v));
    }
    static __device__ __forceinline__ uint16_t narrow1(float v) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    }
    static __device__ __forceinline__ void widen(u32x4 v, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // a copy first: the builtin takes an element's address as the vector's
            const uint32_t w = v[i];
            const f16x2 p = __builtin_bit_cast(f16x2, w);
            f[2 * i] = static_cast<float>(p.x);
            f[2 * i + 1] = static_cast<float>(p.y);
        }
    }
    static __device__ __forceinline__ u32x4 narrow(const float (&f)[8]) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f16x2 p;
            p.x = static_cast<_Float16>(f[2 * i]);
            p.y = static_cast<_Float16>(f[2 * i + 1]);
            v[i] = __builtin_bit_cast(uint32_t, p);
        }
        return v;
    }
};

template <>
struct Wide<BF16> {
    static __device__ __forceinline__ float widen1(uint16_t v) {
        return __builtin_bit_cast(float, static_cast<uint32_t>(v) << 16);
    }
    static __device__ __forceinline__ uint16_t narrow1(float v) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    }
    static __device__ __forceinline__ void widen(u32x4 v, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
            f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ u32x4 narrow(const float (&f)[8]) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bf16x2 p;
            p.x = static_cast<__bf16>(f[2 * i]);
            p.y = static_cast<__bf16>(f[2 * i + 1]);
            v[i] = __builtin_bit_cast(uint32_t, p);
        }
        return v;
    }
};

// NT: non-temporal, for what passes through once and would only push other
// lines out of the caches.  Dirty lines cost twice: a call that leaves them
// behind makes the next call's reads wait for their write-back.
template <bool NT>
__device__ __forceinline__ u32x4 load_vec(const void *p) {
    if constexpr (NT)
        return __builtin_nontemporal_load(static_cast<const u32x4_byte *>(p));
    else
        return *static_cast<const u32x4_byte *>(p);
}

template <bool NT>
__device__ __forceinline__ void store_vec(u32x4 v, void *p) {
    if constexpr (NT)
        __builtin_nontemporal_store(v, static_cast<u32x4_byte *>(p));
    else
        *static_cast<u32x4_byte *>(p) = v;
}

// Where unit i of a row of n values lies.  The last unit of a row that is not
// a whole number of units (TAIL) starts 8 values before the row's end: its
// first `skip` values belong to its neighbour too.  So every unit is one
// access, with nothing to put together value by value (a row of fewer than 8
// values excepted), and both owners compute the same values for what they
// share; only sums have to leave it out.
// Offsets are unsigned 32-bit: added to a wave-uniform row address they need
// one register.
template <bool TAIL>
struct Unit {
    uint32_t start;
    int skip, n;
    __device__ __forceinline__ Unit(int i, int n) : start(8u * i), skip(0), n(n) {
        if constexpr (TAIL) {
            if (8 * i + 8 > n && n >= 8) {
                start = n - 8;
                skip = 8 * i + 8 - n;
            }
        }
    }
    // Value e of the unit is this unit's own.
    __device__ __forceinline__ bool own(int e) const { return !TAIL || (e >= skip && static_cast<int>(start) + e < n); }

    template <bool NT = false>
    __device__ __forceinline__ u32x4 load(const uint16_t *row) const {
        if (!TAIL || n >= 8) return load_vec<NT>(reinterpret_cast<const char *>(row) + 2u * start);
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 7; ++e) v[e / 2] |= e < n ? static_cast<uint32_t>(row[e]) << (16 * (e & 1)) : 0u;
        return v;
    }
    // The whole unit: where no other thread still reads what it shares.
    template <bool NT = false>
    __device__ __forceinline__ void store(uint16_t *row, u32x4 v) const {
        if (!TAIL || n >= 8)
            store_vec<NT>(v, reinterpret_cast<char *>(row) + 2u * start);
        else
            store_own<false>(row, v);
    }
    // The unit's own values.
    template <bool NT = false>
    __device__ __forceinline__ void store_own(uint16_t *row, u32x4 v) const {
        if (!TAIL || (n >= 8 && skip == 0)) {
            store_vec<NT>(v, reinterpret_cast<char *>(row) + 2u * start);
            return;
        }
        // n % 8 values, in pieces of 4, 2 and 1
        uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
        const int rest = n & 7, drop = n >= 8 ? 16 * (8 - rest) : 0;
        if (drop >= 64) {
            lo = hi >> (drop - 64);
        } else if (drop > 0) {
            lo = lo >> drop | hi << (64 - drop);
            hi >>= drop;
        }
        char *p = reinterpret_cast<char *>(row) + 2u * (n - rest);
        if (rest & 4) {
            *reinterpret_cast<u32x2_row *>(p) = u32x2{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32)};
            lo = hi;
            p += 8;
        }
        if (rest & 2) {
            *reinterpret_cast<u32_row *>(p) = static_cast<uint32_t>(lo);
            lo >>= 32;
            p += 4;
        }
        if (rest & 1) *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(lo);
    }
};

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 0x1p-126f;

// The scale of values whose largest magnitude is m (NaN stays NaN).
__device__ __forceinline__ float e4m3_scale(float m) { return m < kE4m3Max * kMinScale ? kMinScale : m / kE4m3Max; }

// y / scale, rounded once, with one reciprocal for the group.  The product
// with it is up to 1.5 units in the last place off, which moves quotients
// half way between two codes.  A step by the remainder brings it within
// one unit, and from there the next gives the division's own result
// (Markstein 1990: a quotient within a unit, the reciprocal to nearest, an
// exact remainder; the negated one keeps the sign of a zero).  Remainders
// are exact for scales from 2^-90 on where a quotient is 2^-11 or more,
// and smaller ones have the code 0; smaller scales are lifted.  What is
// finite over an infinite scale is 0.  (A norm of 16384 x 4096, one contribution
// and a residual, 78.8 us, 84.0 with divisions, 77.6 with the bare product.)
struct E4m3Codes {
    float divisor, inv;
    __device__ __forceinline__ E4m3Codes(float scale, float (&y)[8]) : divisor(scale) {
        if (scale < 0x1p-90f) {
            divisor *= 0x1p60f;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= 0x1p60f;
        }
        inv = 1.0f / divisor;
        divisor = divisor == INFINITY ? 0.0f : divisor;
    }
    __device__ __forceinline__ float over(float v) const {
        float r = v * inv;
        r = fmaf(-fmaf(r, divisor, -v), inv, r);
        return fmaf(-fmaf(r, divisor, -v), inv, r);
    }
    // The codes of the 8 values that the constructor was given.
    __device__ __forceinline__ u32x2 codes(const float (&y)[8]) const {
        u32x2 c;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(over(y[4 * q]), over(y[4 * q + 1]), 0, false);
            v = __builtin_amdgcn_cvt_pk_fp8_f32(over(y[4 * q + 2]), over(y[4 * q + 3]), v, true);
            c[q] = static_cast<uint32_t>(v);
        }
        return c;
    }
};

// Reductions over groups of L consecutive lanes (L a power of two up to 64),
// every lane receiving the result: data-parallel primitives inside a row of
// 16 lanes, lane-row swaps beyond.  The tree is fixed, so sums are the same
// in every run.
// (Every lane has a source in the patterns below, so the value for lanes
// without one does not matter; 0 lets the compiler fold the move into the
// operation that follows.)
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}

template <int L, class T, class F>
__device__ __forceinline__ T reduce_lanes(T v, F f) {
    static_assert(sizeof(T) == 4, "one register");
    auto bits = [](T x) { return __builtin_bit_cast(uint32_t, x); };
    auto back = [](uint32_t x) { return __builtin_bit_cast(T, x); };
    if constexpr (L >= 2) v = f(v, back(dpp<0xB1>(bits(v))));     // lanes 1 0 3 2
    if constexpr (L >= 4) v = f(v, back(dpp<0x4E>(bits(v))));     // lanes 2 3 0 1
    if constexpr (L >= 8) v = f(v, back(dpp<0x141>(bits(v))));    // half rows mirrored
    if constexpr (L >= 16) v = f(v, back(dpp<0x140>(bits(v))));   // rows mirrored
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
        v = f(back(r[0]), back(r[1]));
    }
    if constexpr (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
        v = f(back(r[0]), back(r[1]));
    }
    return v;
}

template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
    return reduce_lanes<L>(v, [](float a, float b) { return a + b; });
}

template <int L>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
    return reduce_lanes<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

__device__ __forceinline__ uint32_t max_of_group(uint32_t v, int lanes) {
    if (lanes == 16) return max_lanes<16>(v);
    if (lanes == 8) return max_lanes<8>(v);
    return max_lanes<4>(v);
}

// A 2-D buffer as a caller passes it: `rows` rows of `width` bytes, `stride`
// bytes apart.
struct Region {
    const void *p;
    size_t rows, width, stride;
};

// True when the two buffers share a byte.  Interleaved columns of one buffer
// (equal strides, disjoint columns) do not.
inline bool regions_overlap(const Region &a, const Region &b) {
    if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t xe = x + (a.rows - 1) * a.stride + a.width, ye = y + (b.rows - 1) * b.stride + b.width;
    if (xe <= y || ye <= x) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
        const size_t d = x < y ? (y - x) % a.stride : (a.stride - (x - y) % a.stride) % a.stride;
        // b's columns start d bytes after a's: apart when they end before the
        // next row's a and begin after this row's
        if (d >= a.width && a.stride - d >= b.width) return false;
    }
    return true;
}

// The same buffer, element for element.
inline bool regions_same(const Region &a, const Region &b) {
    return a.p == b.p && a.rows == b.rows && a.width == b.width && (a.rows <= 1 || a.stride == b.stride);
}

// A row stride in values: 0 stands for contiguous rows.  False when rows
// would overlap or the last byte lies past the address space.
inline bool row_stride(size_t rows, size_t width, size_t *stride, size_t bytes) {
    if (*stride == 0) *stride = width;
    if (rows > 1 && *stride < width) return false;
    size_t span = 0;
    return !__builtin_mul_overflow(rows, *stride, &span) && !__builtin_mul_overflow(span, bytes, &span) &&
           span <= SIZE_MAX / 2;
}

}  // namespace hr
