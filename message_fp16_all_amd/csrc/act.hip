// act.hip -- hr_experts_act_f16 / _bf16: silu(gate) * up between the experts'
// products (or the rows as they are), in 16 bits, in e4m3 with scales, or both;
// and the gradient hr_experts_act_grad_f16 / _bf16.
//
//   s = 1 / (1 + e^-gate)
//   y = gate * s * up
//   dgate = dy * up * s * (1 + gate * (1 - s)),   dup = dy * gate * s
//
// Bound by HBM: every value is read once and written once.  65528 x 2048 to bfloat16 125
// us (6.4 TB/s), its gradient 209 (6.4); to e4m3 113-118 (5.7-6.0), where the instructions of
// the sigmoid, the maximum and the exact quotient take most of the time.
#include <type_traits>

#include "rows.h"

namespace hr {

constexpr int kActThreads = 256;

struct ActArgs {
    const uint16_t *x, *dy;
    uint16_t *out, *dx;
    uint8_t *codes;
    float *scales;
    const int32_t *used;                // NULL, or where the number of rows in use lies
    size_t x_stride, dy_stride, out_stride, dx_stride, codes_stride, scales_stride;
    uint32_t rows;
    int width;
    int group_lanes;
};

// s = 1 / (1 + e^-g) and 1 - s, s to 3 units of 2^-23: the exponential's 1, 1/2 of
// correcting its exponent by all that rounding left out of g log2(e), the sum's 1/2
// and the reciprocal's 1.  (Without the part of log2(e) that binary32 leaves out the
// activation's value was up to 11 units off at a gate of -83; with it 4.5 at most, and
// 65528 x 2048 to e4m3 takes 117.5 us where it took 115.6.)
//
// NEAR (|g| below kNear): from z = e^-g; 1 + z stays in binary32's range.
//
// Otherwise: from z = e^-|g|.  The s of a negative gate soon leaves binary32, and is
// given times 2^64, with `factor` 2^-64 for one of its partners; bfloat16 results are
// still normal.  A near gate that comes this way, because its neighbours are not near,
// is given as the other way gives it: a value's result does not depend on its neighbours.
constexpr float kNear = 87.0f;

template <bool NEAR>
struct Sigmoid {
    float s, rest, factor;
    __device__ __forceinline__ explicit Sigmoid(float g) {
        constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;      // log2(e) = their sum
        constexpr float kLn2 = 0.693147181f;
        if constexpr (NEAR) {
            const float t = g * -kLog2e;
            const float lost = fmaf(g, -kLog2eRest, fmaf(g, -kLog2e, -t));
            float z = __builtin_amdgcn_exp2f(t);
            z = fmaf(z, kLn2 * lost, z);
            s = __builtin_amdgcn_rcpf(1.0f + z);
            rest = z * s;
            factor = 1.0f;
        } else {
            // (64 - t of the rounded t, whose remainder is put right below: fused with
            // the product before, it made values up to 45 units of 2^-23 off)
#pragma clang fp contract(off)
            const float a = fabsf(g);
            const float t = a * kLog2e;
            // (an infinite exponent has no remainder)
            const float lost = t < INFINITY ? fmaf(a, kLog2eRest, fmaf(a, kLog2e, -t)) : 0.0f;
            const bool low = g < 0.0f;
            float z = __builtin_amdgcn_exp2f(low ? 64.0f - t : -t);
            z = fmaf(z, -kLn2 * lost, z);
            factor = low ? 0x1p-64f : 1.0f;
            const float inv = __builtin_amdgcn_rcpf(1.0f + (low ? 0.0f : z));
            const float other = z * inv;
            s = g < 0.0f ? other : inv;
            rest = g < 0.0f ? inv : other;
            if (g != g) s = rest = g;
            if (a < kNear) {
                const Sigmoid<true> near(g);
                s = near.s, rest = near.rest, factor = 1.0f;
            }
        }
    }
};

// Whether all of the wave's gates are near: which is nearly always so, and makes a
// value's sigmoid 9 instructions instead of some 20.
__device__ __forceinline__ bool all_near(const float (&g)[8]) {
    bool near = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) near = near && fabsf(g[e]) < kNear;
    return __all(near);
}

__device__ __forceinline__ uint32_t rows_used(const ActArgs &a) {
    if (a.used == nullptr) return a.rows;
    const int n = *a.used;
    return n < 0 ? 0u : static_cast<uint32_t>(n) < a.rows ? static_cast<uint32_t>(n) : a.rows;
}

// L lanes per row, a unit of 8 values of U rows each at a time, so that a lane has
// 2 U loads on their way before it works on the first.
template <class E, int L, int U, bool GATED, bool TAIL, bool NT>
__global__ __launch_bounds__(kActThreads) void act_rows(ActArgs a) {
    constexpr uint32_t R = kActThreads / L;
    const uint32_t used = rows_used(a);
    const uint32_t r0 = blockIdx.x * (R * U) + threadIdx.x / L;
    if (blockIdx.x * (R * U) >= used) return;
    const int lane = static_cast<int>(threadIdx.x) % L, units = (a.width + 7) / 8;
    // (every lane of a group takes part in its maximum)
    for (int i0 = 0; i0 < units; i0 += L) {
        const int i = i0 + lane;
        const Unit<TAIL> at(i < units ? i : 0, a.width);
        u32x4 in[U], up[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t r = r0 + u * R;
            in[u] = up[u] = u32x4{0, 0, 0, 0};
            if (r < used && i < units) {
                const uint16_t *x = a.x + r * a.x_stride;
                in[u] = at.template load<NT>(x);
                if constexpr (GATED) up[u] = at.template load<NT>(x + a.width);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t r = r0 + u * R;
            const bool there = r < used && i < units;
            float y[8];
            Wide<E>::widen(in[u], y);
            if constexpr (GATED) {
                float v[8];
                Wide<E>::widen(up[u], v);
                const auto gate = [&](auto near) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const Sigmoid<decltype(near)::value> g(y[e]);
                        y[e] = y[e] * g.s * (v[e] * g.factor);
                    }
                };
                if (all_near(y))
                    gate(std::true_type());
                else
                    gate(std::false_type());
            }
            if (there && a.out != nullptr) at.template store_own<NT>(a.out + r * a.out_stride, Wide<E>::narrow(y));
            if (a.codes == nullptr) continue;
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = __builtin_bit_cast(uint32_t, y[e]) & 0x7FFFFFFFu;
                if (there && at.own(e)) top = m > top ? m : top;
            }
            top = max_of_group(top, a.group_lanes);
            if (!there) continue;
            const float scale = e4m3_scale(__builtin_bit_cast(float, top));
            if (i % a.group_lanes == 0) a.scales[r * a.scales_stride + i / a.group_lanes] = scale;
            const E4m3Codes at_scale(scale, y);
            const u32x2 c = at_scale.codes(y);
            uint8_t *p = a.codes + r * a.codes_stride + at.start;
            if (!TAIL || (a.width >= 8 && at.skip == 0)) {
                if constexpr (NT)
                    __builtin_nontemporal_store(c, reinterpret_cast<u32x2_row *>(p));
                else
                    *reinterpret_cast<u32x2_row *>(p) = c;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at.own(e)) p[e] = static_cast<uint8_t>(c[e / 4] >> (8 * (e & 3)));
            }
        }
    }
}

template <class E, int L, int U, bool TAIL, bool NT>
__global__ __launch_bounds__(kActThreads) void act_grad_rows(ActArgs a) {
    constexpr uint32_t R = kActThreads / L;
    const uint32_t used = rows_used(a);
    const uint32_t r0 = blockIdx.x * (R * U) + threadIdx.x / L;
    if (r0 >= used) return;
    const int lane = static_cast<int>(threadIdx.x) % L, units = (a.width + 7) / 8;
    for (int i = lane; i < units; i += L) {
        // (dx may be x: a unit's values that are its neighbour's may have been
        // overwritten, and are not stored)
        const Unit<TAIL> at(i, a.width);
        u32x4 in[3][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t r = r0 + u * R;
            if (r < used) {
                const uint16_t *x = a.x + r * a.x_stride;
                in[0][u] = at.template load<NT>(x);
                in[1][u] = at.template load<NT>(x + a.width);
                in[2][u] = at.template load<NT>(a.dy + r * a.dy_stride);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t r = r0 + u * R;
            if (r >= used) continue;
            uint16_t *dx = a.dx + r * a.dx_stride;
            float gate[8], up[8], d[8], y[8];
            Wide<E>::widen(in[0][u], gate);
            Wide<E>::widen(in[1][u], up);
            Wide<E>::widen(in[2][u], d);
            const auto grad = [&](auto near) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const Sigmoid<decltype(near)::value> g(gate[e]);
                    const float silu = gate[e] * g.s;
                    const float v = up[e] * g.factor;
                    y[e] = silu * v;
                    up[e] = d[e] * v * (g.s * fmaf(gate[e], g.rest, 1.0f));
                    gate[e] = d[e] * g.factor * silu;
                }
            };
            if (all_near(gate))
                grad(std::true_type());
            else
                grad(std::false_type());
            at.template store_own<NT>(dx, Wide<E>::narrow(up));
            at.template store_own<NT>(dx + a.width, Wide<E>::narrow(gate));
            if (a.out != nullptr) at.template store_own<NT>(a.out + r * a.out_stride, Wide<E>::narrow(y));
        }
    }
}

namespace {

int act_lanes(size_t width) { return width <= 128 ? 16 : width <= 512 ? 64 : kActThreads; }

// Calls that read or write this much go past the caches, two rows to a lane.
// Measured from three sets of buffers in turn, one row cached and two streamed:
// activation 65528 x 2048 to bfloat16 135 and 127 us, as rows are to e4m3 77 and 63,
// gradient 234 and 209; of 16383 x 4096 143 and 135; 8192 x 2048 to e4m3 (101 MB) 19.2
// and 20.6, its gradient (168 MB) 30.9 and 28.3; four rows 130, 65, 218, 141.
constexpr size_t kActStreamBytes = size_t(1) << 27;
constexpr int kActRows = 2;

template <class K>
hr_status launch_act(K kernel, int lanes, int rows, const ActArgs &a, hr_stream_t stream) {
    const size_t high = static_cast<size_t>(kActThreads / lanes) * rows;
    const size_t grid = (a.rows + high - 1) / high;
    if (grid >= (size_t(1) << 32) / kActThreads) return HR_ERR_TOO_LARGE;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(kActThreads), 0,
                       reinterpret_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? HR_OK : HR_ERR_HIP;
}

// The variant of a kernel K<E, lanes, rows, .., TAIL, NT> for a call: several rows to
// a lane, past the caches, where the values are many.
#define HR_ACT_AT(K, L, U, NT, ...)                                                                       \
    (a.width % 8 != 0 ? launch_act(K<E, L, U, ##__VA_ARGS__, true, NT>, L, U, a, stream)                    \
                      : launch_act(K<E, L, U, ##__VA_ARGS__, false, NT>, L, U, a, stream))
#define HR_ACT(K, ...)                                                                                    \
    do {                                                                                                  \
        const int lanes = act_lanes(a.width);                                                             \
        if (static_cast<size_t>(a.rows) * a.width * (a.dy != nullptr ? 10 : 4) >= kActStreamBytes) {                               \
            if (lanes == 16) return HR_ACT_AT(K, 16, kActRows, true, ##__VA_ARGS__);                      \
            if (lanes == 64) return HR_ACT_AT(K, 64, kActRows, true, ##__VA_ARGS__);                      \
            return HR_ACT_AT(K, kActThreads, kActRows, true, ##__VA_ARGS__);                              \
        }                                                                                                 \
        if (lanes == 16) return HR_ACT_AT(K, 16, 1, false, ##__VA_ARGS__);                                \
        if (lanes == 64) return HR_ACT_AT(K, 64, 1, false, ##__VA_ARGS__);                                \
        return HR_ACT_AT(K, kActThreads, 1, false, ##__VA_ARGS__);                                        \
    } while (0)

template <class E, bool GATED>
hr_status run_act(const ActArgs &a, hr_stream_t stream) {
    HR_ACT(act_rows, GATED);
}

template <class E>
hr_status run_act_grad(const ActArgs &a, hr_stream_t stream) {
    HR_ACT(act_grad_rows);
}

#undef HR_ACT
#undef HR_ACT_AT

template <class E>
hr_status act_impl(const hr_experts_act_args *q, hr_stream_t stream) {
    if (q == nullptr || q->width == 0 || (q->codes == nullptr) != (q->scales == nullptr) ||
        (q->offsets != nullptr && q->experts < 1))
        return HR_ERR_INVALID_ARG;
    if (q->codes != nullptr && q->group != 32 && q->group != 64 && q->group != 128) return HR_ERR_INVALID_ARG;
    if (q->rows > 0x7FFFFFFFu || q->width > HR_EXPERTS_PRODUCT_MAX) return HR_ERR_TOO_LARGE;
    const size_t in = q->gated ? 2 * q->width : q->width;
    const size_t groups = q->codes != nullptr ? (q->width + q->group - 1) / q->group : 1;
    ActArgs a{};
    a.x_stride = q->x_stride;
    a.out_stride = q->out_stride;
    a.codes_stride = q->codes_stride;
    a.scales_stride = q->scales_stride;
    if (!row_stride(q->rows, in, &a.x_stride, 2) || !row_stride(q->rows, q->width, &a.out_stride, 2) ||
        !row_stride(q->rows, q->width, &a.codes_stride, 1) || !row_stride(q->rows, groups, &a.scales_stride, 4))
        return HR_ERR_INVALID_ARG;
    if (q->rows == 0) return HR_OK;
    if (q->x == nullptr || (q->out == nullptr && q->codes == nullptr)) return HR_ERR_INVALID_ARG;
    if (!aligned(q->x, 2) || !aligned(q->out, 2) || !aligned(q->scales, 4) || !aligned(q->offsets, 4))
        return HR_ERR_ALIGNMENT;
    const Region ins[] = {{q->x, q->rows, in * 2, a.x_stride * 2},
                          {q->offsets, 1, (static_cast<size_t>(q->experts > 0 ? q->experts : 0) + 1) * 4, 0}};
    const Region outs[] = {{q->out, q->rows, q->width * 2, a.out_stride * 2},
                           {q->codes, q->rows, q->width, a.codes_stride},
                           {q->scales, q->rows, groups * 4, a.scales_stride * 4}};
    for (int i = 0; i < 3; ++i) {
        for (const Region &r : ins)
            if (regions_overlap(outs[i], r)) return HR_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (regions_overlap(outs[i], outs[j])) return HR_ERR_INVALID_ARG;
    }
    a.x = static_cast<const uint16_t *>(q->x);
    a.out = static_cast<uint16_t *>(q->out);
    a.codes = static_cast<uint8_t *>(q->codes);
    a.scales = q->scales;
    a.used = q->offsets != nullptr ? q->offsets + q->experts : nullptr;
    a.rows = static_cast<uint32_t>(q->rows);
    a.width = static_cast<int>(q->width);
    a.group_lanes = q->group / 8;
    return q->gated ? run_act<E, true>(a, stream) : run_act<E, false>(a, stream);
}

template <class E>
hr_status act_grad_impl(const hr_experts_act_grad_args *q, hr_stream_t stream) {
    if (q == nullptr || q->width == 0 || (q->offsets != nullptr && q->experts < 1)) return HR_ERR_INVALID_ARG;
    if (q->rows > 0x7FFFFFFFu || q->width > HR_EXPERTS_PRODUCT_MAX) return HR_ERR_TOO_LARGE;
    const size_t w = q->width;
    ActArgs a{};
    a.dy_stride = q->dy_stride;
    a.x_stride = q->x_stride;
    a.dx_stride = q->dx_stride;
    a.out_stride = q->out_stride;
    if (!row_stride(q->rows, w, &a.dy_stride, 2) || !row_stride(q->rows, 2 * w, &a.x_stride, 2) ||
        !row_stride(q->rows, 2 * w, &a.dx_stride, 2) || !row_stride(q->rows, w, &a.out_stride, 2))
        return HR_ERR_INVALID_ARG;
    if (q->rows == 0) return HR_OK;
    if (q->x == nullptr || q->dy == nullptr || q->dx == nullptr) return HR_ERR_INVALID_ARG;
    if (!aligned(q->x, 2) || !aligned(q->dy, 2) || !aligned(q->dx, 2) || !aligned(q->out, 2) || !aligned(q->offsets, 4))
        return HR_ERR_ALIGNMENT;
    const Region x = {q->x, q->rows, w * 4, a.x_stride * 2}, dy = {q->dy, q->rows, w * 2, a.dy_stride * 2};
    const Region dx = {q->dx, q->rows, w * 4, a.dx_stride * 2}, out = {q->out, q->rows, w * 2, a.out_stride * 2};
    const Region offsets = {q->offsets, 1, (static_cast<size_t>(q->experts > 0 ? q->experts : 0) + 1) * 4, 0};
    if (regions_overlap(dx, dy) || regions_overlap(dx, offsets) || regions_overlap(out, x) || regions_overlap(out, dy) ||
        regions_overlap(out, dx) || regions_overlap(out, offsets) || (regions_overlap(dx, x) && !regions_same(dx, x)))
        return HR_ERR_INVALID_ARG;
    a.x = static_cast<const uint16_t *>(q->x);
    a.dy = static_cast<const uint16_t *>(q->dy);
    a.dx = static_cast<uint16_t *>(q->dx);
    a.out = static_cast<uint16_t *>(q->out);
    a.used = q->offsets != nullptr ? q->offsets + q->experts : nullptr;
    a.rows = static_cast<uint32_t>(q->rows);
    a.width = static_cast<int>(w);
    return run_act_grad<E>(a, stream);
}

}  // namespace
}  // namespace hr

extern "C" {

hr_status hr_experts_act_f16(const hr_experts_act_args *args, hr_stream_t stream) {
    return hr::act_impl<hr::F16>(args, stream);
}
hr_status hr_experts_act_bf16(const hr_experts_act_args *args, hr_stream_t stream) {
    return hr::act_impl<hr::BF16>(args, stream);
}
hr_status hr_experts_act_grad_f16(const hr_experts_act_grad_args *args, hr_stream_t stream) {
    return hr::act_grad_impl<hr::F16>(args, stream);
}
hr_status hr_experts_act_grad_bf16(const hr_experts_act_grad_args *args, hr_stream_t stream) {
    return hr::act_grad_impl<hr::BF16>(args, stream);
}

}  // extern "C"
