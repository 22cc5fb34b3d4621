// product_call.h -- checks of the experts' products' arguments and the choice
// of a kernel; not exported.
#pragma once

#include "product.h"
#include "product_shape.h"

namespace hr {

// Rows of at most 4 MiB apart: a tile's 256 stay inside a buffer's 2 GiB.  (One
// row has no other to be apart from.)
constexpr size_t kMaxProductStride = size_t(1) << 22;
inline bool too_far_apart(size_t rows, size_t bytes) { return rows > 1 && bytes > kMaxProductStride; }
// A row number and some stages' rows behind it stay below 2^31.
constexpr size_t kMaxProductRows = (size_t(1) << 31) - 4096;

inline bool units16(const void *p) { return aligned(p, 16); }

// Matrices of `rows` rows of `width` values, as a caller passes them.
struct Matrices {
    size_t stride, expert_stride;       // values
    Region region;
};
inline bool matrices(const void *p, int experts, size_t rows, size_t width, size_t stride, size_t expert_stride,
                     size_t bytes, Matrices *m) {
    m->stride = stride;
    if (!row_stride(rows, width, &m->stride, bytes)) return false;
    m->expert_stride = expert_stride;
    const size_t span = rows * m->stride;               // below 2^63: checked
    if (m->expert_stride == 0) m->expert_stride = span;
    if (experts > 1 && m->expert_stride < (rows - 1) * m->stride + width) return false;
    size_t all = 0;
    if (__builtin_mul_overflow(static_cast<size_t>(experts), m->expert_stride, &all) ||
        __builtin_mul_overflow(all, bytes, &all) || all > SIZE_MAX / 2)
        return false;
    if (experts == 1 || m->expert_stride == span)
        m->region = {p, static_cast<size_t>(experts) * rows, width * bytes, m->stride * bytes};
    else
        m->region = {p, static_cast<size_t>(experts), ((rows - 1) * m->stride + width) * bytes,
                     m->expert_stride * bytes};
    return true;
}

template <int SIZE>
hr_status product_check(const hr_experts_product_args *q, ProductArgs &a, bool &any) {
    if (q == nullptr || q->n == 0 || q->k == 0 || q->experts < 1 || (q->offsets == nullptr && q->experts != 1))
        return HR_ERR_INVALID_ARG;
    if (q->n > HR_EXPERTS_PRODUCT_MAX || q->k > HR_EXPERTS_PRODUCT_MAX || q->experts > HR_EXPERTS_MAX ||
        q->rows > kMaxProductRows)
        return HR_ERR_TOO_LARGE;
    const bool across = q->transposed != 0;
    const size_t wr = across ? q->k : q->n, wc = across ? q->n : q->k;
    size_t xs = q->x_stride, os = q->out_stride, ss = q->x_scales_stride;
    Matrices w, ws{};
    const size_t kb = (q->k + 127) / 128, rb = (wr + 127) / 128, cb = (wc + 127) / 128;
    if (!row_stride(q->rows, q->k, &xs, SIZE) || !row_stride(q->rows, q->n, &os, 2) ||
        !matrices(q->w, q->experts, wr, wc, q->w_stride, q->w_expert_stride, SIZE, &w))
        return HR_ERR_INVALID_ARG;
    if (SIZE == 1 && (!row_stride(q->rows, kb, &ss, 4) ||
                      !matrices(q->w_scales, q->experts, rb, cb, q->w_scales_stride, q->w_scales_expert_stride, 4, &ws)))
        return HR_ERR_INVALID_ARG;
    if (too_far_apart(q->rows, xs * SIZE) || too_far_apart(wr, w.stride * SIZE) || too_far_apart(q->rows, os * 2) ||
        (SIZE == 1 && too_far_apart(q->rows, ss * 4)))
        return HR_ERR_TOO_LARGE;
    if (q->rows == 0) return HR_OK;
    if (q->x == nullptr || q->w == nullptr || q->out == nullptr) return HR_ERR_INVALID_ARG;
    if (SIZE == 1 && (q->x_scales == nullptr || q->w_scales == nullptr)) return HR_ERR_INVALID_ARG;
    if (!aligned(q->x, SIZE) || !aligned(q->w, SIZE) || !aligned(q->out, 2) || !aligned(q->offsets, 4) ||
        !aligned(q->x_scales, 4) || !aligned(q->w_scales, 4))
        return HR_ERR_ALIGNMENT;
    const Region out = {q->out, q->rows, q->n * 2, os * 2};
    if (regions_overlap(out, {q->x, q->rows, q->k * SIZE, xs * SIZE}) || regions_overlap(out, w.region) ||
        regions_overlap(out, {q->offsets, 1, (static_cast<size_t>(q->experts) + 1) * 4, 0}))
        return HR_ERR_INVALID_ARG;
    if (SIZE == 1 && (regions_overlap(out, {q->x_scales, q->rows, kb * 4, ss * 4}) || regions_overlap(out, ws.region)))
        return HR_ERR_INVALID_ARG;
    a.q = static_cast<const char *>(q->x);
    a.p = static_cast<const char *>(q->w);
    a.out = static_cast<char *>(q->out);
    a.offsets = q->offsets;
    a.q_scales = q->x_scales;
    a.p_scales = q->w_scales;
    a.q_stride = xs * SIZE;
    a.p_stride = w.stride * SIZE;
    a.out_stride = os * 2;
    a.p_expert_stride = w.expert_stride * SIZE;
    a.q_scales_stride = ss;
    a.scales_expert = ws.expert_stride;
    a.scales_p = across ? 1 : ws.stride;
    a.scales_c = across ? ws.stride : 1;
    a.rows = static_cast<uint32_t>(q->rows);
    a.experts = q->experts;
    a.np = static_cast<int>(q->n);
    a.nc = static_cast<int>(q->k);
    // DMA brings whole 16-byte units from 16-byte addresses
    any = !(units16(q->x) && units16(q->w) && a.q_stride % 16 == 0 && a.p_stride % 16 == 0 &&
            a.p_expert_stride % 16 == 0 && q->k * SIZE % 16 == 0 && (!across || q->n * SIZE % 16 == 0));
    return HR_OK;
}

inline hr_status product_grad_check(const hr_experts_product_grad_args *q, ProductArgs &a, bool &any) {
    if (q == nullptr || q->n == 0 || q->k == 0 || q->experts < 1 || (q->offsets == nullptr && q->experts != 1))
        return HR_ERR_INVALID_ARG;
    if (q->n > HR_EXPERTS_PRODUCT_MAX || q->k > HR_EXPERTS_PRODUCT_MAX || q->experts > HR_EXPERTS_MAX ||
        q->rows > kMaxProductRows)
        return HR_ERR_TOO_LARGE;
    size_t ys = q->dy_stride, xs = q->x_stride;
    const size_t ob = q->dw_f32 ? 4 : 2;
    Matrices w;
    if (!row_stride(q->rows, q->n, &ys, 2) || !row_stride(q->rows, q->k, &xs, 2) ||
        !matrices(q->dw, q->experts, q->n, q->k, q->dw_stride, q->dw_expert_stride, ob, &w))
        return HR_ERR_INVALID_ARG;
    if (too_far_apart(q->rows, ys * 2) || too_far_apart(q->rows, xs * 2) || too_far_apart(q->n, w.stride * ob))
        return HR_ERR_TOO_LARGE;
    if (q->dw == nullptr || (q->rows > 0 && (q->dy == nullptr || q->x == nullptr))) return HR_ERR_INVALID_ARG;
    if (!aligned(q->dy, 2) || !aligned(q->x, 2) || !aligned(q->dw, ob) || !aligned(q->offsets, 4))
        return HR_ERR_ALIGNMENT;
    if (regions_overlap(w.region, {q->dy, q->rows, q->n * 2, ys * 2}) ||
        regions_overlap(w.region, {q->x, q->rows, q->k * 2, xs * 2}) ||
        regions_overlap(w.region, {q->offsets, 1, (static_cast<size_t>(q->experts) + 1) * 4, 0}))
        return HR_ERR_INVALID_ARG;
    a.q = static_cast<const char *>(q->dy);
    a.p = static_cast<const char *>(q->x);
    a.out = static_cast<char *>(q->dw);
    a.offsets = q->offsets;
    a.q_stride = ys * 2;
    a.p_stride = xs * 2;
    a.out_stride = w.stride * ob;
    a.out_expert_stride = w.expert_stride * ob;
    a.rows = static_cast<uint32_t>(q->rows);
    a.experts = q->experts;
    a.nq = static_cast<int>(q->n);
    a.np = static_cast<int>(q->k);
    // (as the expert rows': dw of 1.07 GB 816 us, past the caches 742; of 134 MB 35 and 47)
    a.stream = w.region.rows * w.region.width >= size_t(1) << 28;
    any = !(units16(q->dy) && units16(q->x) && a.q_stride % 16 == 0 && a.p_stride % 16 == 0 && q->n % 8 == 0 &&
            q->k % 8 == 0);
    return HR_OK;
}

template <class K>
hr_status launch_tiles(K kernel, size_t tiles, int threads, hr_stream_t stream, const ProductArgs &a) {
    // (the dies' shares of the tiles are rounded up; a launch has fewer than 2^32 work-items)
    const size_t grid = (tiles + 7) / 8 * 8;
    if (grid >= (size_t(1) << 32) / threads) return HR_ERR_TOO_LARGE;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, reinterpret_cast<hipStream_t>(stream),
                       a);
    return hipGetLastError() == hipSuccess ? HR_OK : HR_ERR_HIP;
}

// One workgroup of large tiles per compute unit, as many to each of the eight dies.
template <class K>
hr_status launch_large(K kernel, size_t tiles, hr_stream_t stream, const ProductArgs &a) {
    if (tiles >= size_t(1) << 31) return HR_ERR_TOO_LARGE;
    int device = 0, units = 0;
    if (stream_device(stream, &device) != hipSuccess || device_cu_count(device, &units) != hipSuccess) return HR_ERR_HIP;
    const size_t most = units < 8 ? 8 : static_cast<size_t>(units) / 8 * 8;
    return launch_tiles(kernel, tiles < most ? tiles : most, 512, stream, a);
}

// The shapes, from the largest: tile, waves over q, p and the panels of a stage,
// stages.  Where weights are read for few rows all but the smallest come near to
// HBM's rate, and what counts is that the GPU is full.
typedef Shape<128, 256, 2, 4, 1, 3> Half;
typedef Shape<128, 128, 2, 2, 1, 2, 2> Middle;
typedef Shape<64, 128, 2, 2, 1, 3, 2> Some;
typedef Shape<32, 128, 1, 2, 2, 3> Low;
typedef Shape<16, 32, 1, 1, 4, 3, 2> Few;
typedef Shape<16, 64, 1, 1, 4, 3> FewAcross;    // (32 values of a strided row are half a line)
typedef Shape<16, 16, 1, 1, 4, 4> Tiny;
typedef Shape<64, 64, 1, 1, 4, 2> Deep;         // the gradient of few matrices
typedef Shape<16, 32, 1, 1, 4, 2, 3> AnyFew;

template <class E, class O, class SH, bool PA, bool ANY>
hr_status run_product(ProductArgs &a, hr_stream_t stream) {
    a.tiles_p = (a.np + SH::BP - 1) / SH::BP;
    return launch_tiles(product_tiles<E, O, SH, false, PA, false, ANY>, tiles_of(a.rows, a.experts, SH::BQ) * a.tiles_p,
                        SH::kThreads, stream, a);
}

template <class E, class O, bool PA>
hr_status pick_product(ProductArgs &a, bool any, hr_stream_t stream) {
    const ProductShape shape = product_shape(a.rows, a.experts, a.np, PA, any);
    switch (shape) {
        case ProductShape::Large:
            a.tiles_p = (a.np + 255) / 256;
            return launch_large(product_large<E, O, false, PA, false>, tiles_of(a.rows, a.experts, 256) * a.tiles_p, stream, a);
        case ProductShape::Half: return run_product<E, O, Half, PA, false>(a, stream);
        case ProductShape::Middle: return run_product<E, O, Middle, PA, false>(a, stream);
        case ProductShape::Some: return run_product<E, O, Some, PA, false>(a, stream);
        case ProductShape::Low: return run_product<E, O, Low, PA, false>(a, stream);
        case ProductShape::AnyMiddle: return run_product<E, O, Middle, PA, true>(a, stream);
        case ProductShape::AnyFew: return run_product<E, O, AnyFew, PA, true>(a, stream);
        default: break;                 // the lowest: of one layout each
    }
    if constexpr (PA)
        return run_product<E, O, FewAcross, PA, false>(a, stream);
    else if (shape == ProductShape::Few)
        return run_product<E, O, Few, PA, false>(a, stream);
    else
        return run_product<E, O, Tiny, PA, false>(a, stream);
}

template <class E, class O>
hr_status launch_product(ProductArgs &a, bool across, bool any, hr_stream_t stream) {
    return across ? pick_product<E, O, true>(a, any, stream) : pick_product<E, O, false>(a, any, stream);
}

template <class E, class O, class SH, bool ANY>
hr_status run_product_grad(ProductArgs &a, hr_stream_t stream) {
    a.tiles_q = (a.nq + SH::BQ - 1) / SH::BQ;
    a.tiles_p = (a.np + SH::BP - 1) / SH::BP;
    const size_t each = static_cast<size_t>(a.tiles_q) * a.tiles_p;
    return launch_tiles(product_tiles<E, O, SH, true, true, true, ANY>, each * a.experts, SH::kThreads, stream, a);
}

template <class E, class O>
hr_status launch_product_grad(ProductArgs &a, bool any, hr_stream_t stream) {
    switch (gradient_shape(a.experts, a.nq, a.np, any)) {
        case GradientShape::Large: {
            a.tiles_q = (a.nq + 255) / 256;
            a.tiles_p = (a.np + 255) / 256;
            const size_t tiles = static_cast<size_t>(a.tiles_q) * a.tiles_p * a.experts;
            if (tiles >= size_t(1) << 31) return HR_ERR_TOO_LARGE;
            return launch_large(product_large<E, O, true, true, true>, tiles, stream, a);
        }
        case GradientShape::Middle: return run_product_grad<E, O, Middle, false>(a, stream);
        case GradientShape::AnyMiddle: return run_product_grad<E, O, Middle, true>(a, stream);
        default: return run_product_grad<E, O, Deep, false>(a, stream);
    }
}

}  // namespace hr
