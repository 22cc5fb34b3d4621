// act.hip -- hr_experts_act_f16 / _bf16: silu(gate) * up between the experts'
// products (or the rows as they are), in 16 bits, in e4m3 with scales, or both;
// and the gradient hr_experts_act_grad_f16 / _bf16.
//
//   s = 1 / (1 + e^-gate)
//   y = gate * s * up
//   dgate = dy * up * s * (1 + gate * (1 - s)),   dup = dy * gate * s
//
// Bound by HBM: every value is read once and written once.
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

// s = 1 / (1 + e^-g) and 1 - s, each to a few units in the last place: from
// z = e^-|g|, whose exponent is corrected by what rounding it left out.  Where s
// would leave binary32 (g below -64 ln 2), it is given times 2^64, with
// `factor` 2^-64 for one of its partners; bfloat16 results there are still normal.
struct Sigmoid {
    float s, rest, factor;
    __device__ __forceinline__ explicit Sigmoid(float g) {
        constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;      // log2(e) = their sum
        const float a = fabsf(g);
        const float t = a * kLog2e;
        // (an infinite exponent has no remainder)
        const float lost = t < INFINITY ? fmaf(a, kLog2eRest, fmaf(a, kLog2e, -t)) : 0.0f;
        const bool low = g < 0.0f && t > 64.0f;
        float z = __builtin_amdgcn_exp2f(low ? 64.0f - t : -t);
        z = fmaf(z, -0.693147181f * lost, z);
        factor = low ? 0x1p-64f : 1.0f;
        const float inv = __builtin_amdgcn_rcpf(1.0f + (low ? 0.0f : z));
        const float other = z * inv;
        s = g < 0.0f ? other : inv;
        rest = g < 0.0f ? inv : other;
        if (g != g) s = rest = g;
    }
};

__device__ __forceinline__ uint32_t rows_used(const ActArgs &a) {
    if (a.used == nullptr) return a.rows;
    const int n = *a.used;
    return n < 0 ? 0u : static_cast<uint32_t>(n) < a.rows ? static_cast<uint32_t>(n) : a.rows;
}

// L lanes per row, one unit of 8 values each at a time.
template <class E, int L, bool GATED, bool TAIL>
__global__ __launch_bounds__(kActThreads) void act_rows(ActArgs a) {
    constexpr uint32_t R = kActThreads / L;
    const uint32_t used = rows_used(a);
    const uint32_t r = blockIdx.x * R + threadIdx.x / L;
    if (blockIdx.x * R >= used) return;
    const bool here = r < used;
    const int lane = static_cast<int>(threadIdx.x) % L, units = (a.width + 7) / 8;
    const uint16_t *x = a.x + r * a.x_stride;
    // (every lane of a group takes part in its maximum)
    for (int i0 = 0; i0 < units; i0 += L) {
        const int i = i0 + lane;
        const bool there = here && i < units;
        const Unit<TAIL> at(there ? i : 0, a.width);
        float y[8] = {};
        if (there) {
            Wide<E>::widen(at.load(x), y);
            if constexpr (GATED) {
                float up[8];
                Wide<E>::widen(at.load(x + a.width), up);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const Sigmoid g(y[e]);
                    y[e] = y[e] * g.s * (up[e] * g.factor);
                }
            }
            if (a.out != nullptr) at.store_own(a.out + r * a.out_stride, Wide<E>::narrow(y));
        }
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
            *reinterpret_cast<u32x2_row *>(p) = c;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at.own(e)) p[e] = static_cast<uint8_t>(c[e / 4] >> (8 * (e & 3)));
        }
    }
}

template <class E, int L, bool TAIL>
__global__ __launch_bounds__(kActThreads) void act_grad_rows(ActArgs a) {
    constexpr uint32_t R = kActThreads / L;
    const uint32_t r = blockIdx.x * R + threadIdx.x / L;
    if (r >= rows_used(a)) return;
    const int lane = static_cast<int>(threadIdx.x) % L, units = (a.width + 7) / 8;
    const uint16_t *x = a.x + r * a.x_stride, *dy = a.dy + r * a.dy_stride;
    uint16_t *dx = a.dx + r * a.dx_stride;
    for (int i = lane; i < units; i += L) {
        // (dx may be x: a unit's values that are its neighbour's may have been
        // overwritten, and are not stored)
        const Unit<TAIL> at(i, a.width);
        float gate[8], up[8], d[8], y[8];
        Wide<E>::widen(at.load(x), gate);
        Wide<E>::widen(at.load(x + a.width), up);
        Wide<E>::widen(at.load(dy), d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const Sigmoid g(gate[e]);
            const float silu = gate[e] * g.s;
            const float u = up[e] * g.factor;
            y[e] = silu * u;
            up[e] = d[e] * u * (g.s * fmaf(gate[e], g.rest, 1.0f));
            gate[e] = d[e] * g.factor * silu;
        }
        at.store_own(dx, Wide<E>::narrow(up));
        at.store_own(dx + a.width, Wide<E>::narrow(gate));
        if (a.out != nullptr) at.store_own(a.out + r * a.out_stride, Wide<E>::narrow(y));
    }
}

namespace {

int act_lanes(size_t width) { return width <= 128 ? 16 : width <= 512 ? 64 : kActThreads; }

template <class K>
hr_status launch_act(K kernel, int lanes, const ActArgs &a, hr_stream_t stream) {
    const size_t grid = (static_cast<size_t>(a.rows) + kActThreads / lanes - 1) / (kActThreads / lanes);
    if (grid >= (size_t(1) << 32) / kActThreads) return HR_ERR_TOO_LARGE;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(kActThreads), 0,
                       reinterpret_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? HR_OK : HR_ERR_HIP;
}

template <class E, bool GATED>
hr_status run_act(const ActArgs &a, hr_stream_t stream) {
    const int lanes = act_lanes(a.width);
    const bool tail = a.width % 8 != 0;
    if (lanes == 16) return launch_act(tail ? act_rows<E, 16, GATED, true> : act_rows<E, 16, GATED, false>, 16, a, stream);
    if (lanes == 64) return launch_act(tail ? act_rows<E, 64, GATED, true> : act_rows<E, 64, GATED, false>, 64, a, stream);
    return launch_act(tail ? act_rows<E, kActThreads, GATED, true> : act_rows<E, kActThreads, GATED, false>, kActThreads,
                      a, stream);
}

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
    const int lanes = act_lanes(w);
    const bool tail = w % 8 != 0;
    if (lanes == 16) return launch_act(tail ? act_grad_rows<E, 16, true> : act_grad_rows<E, 16, false>, 16, a, stream);
    if (lanes == 64) return launch_act(tail ? act_grad_rows<E, 64, true> : act_grad_rows<E, 64, false>, 64, a, stream);
    return launch_act(tail ? act_grad_rows<E, kActThreads, true> : act_grad_rows<E, kActThreads, false>, kActThreads, a,
                      stream);
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
