// norm.hip -- hr_reduce_rmsnorm_f16 / _bf16: the fold of G contributions with
// the residual as its last operand, the root-mean-square norm of the sum and
// its output in 16 bits, in e4m3 with scales, or both; and the norm's gradient
// hr_rmsnorm_grad_f16 / _bf16.
//
//   h = fold(x_0, .., x_{G-1}, residual)        16 bits, one rounding per add
//   rstd = 1 / sqrt(mean(h^2) + eps)            binary32
//   y = h * rstd * weight                       binary32, rounded once to out
//   scale = max(max|y| / 448, 2^-126)           over the row or a group of it
//   code = e4m3(y / scale)                      from the unrounded y
//
// h is what hr_reduce_f16 gives for G + 1 contributions, bit for bit, and the
// norm is taken of these 16-bit values, not of an unrounded sum: a residual
// stream kept by this call, by hr_reduce and by an exchange is the same.
#include "rows.h"

namespace hr {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxWaves = kNormMaxThreads / kWave;
constexpr int kOperands = HR_MAX_G + 1;
constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 0x1p-126f;

struct NormArgs {
    const uint16_t *in[kOperands];   // contributions, then the residual if there is one
    const void *weight;
    uint16_t *h;
    uint16_t *out;
    uint8_t *codes;
    float *scales;
    float *rstd;
    size_t rows;
    size_t in_stride, last_stride;   // of in[0 .. n-2] and of in[n-1]
    size_t h_stride, out_stride, codes_stride, scales_stride;
    int n;                           // operands of the fold
    int hidden;
    int weight_f32;
    int group_lanes;                 // lanes (8 values each) that share a scale; 0 = the row
    float eps;
};

// The 8 weights of a unit; values past the row's end are 0, and without a
// weight all are 1.
template <class E, bool TAIL>
__device__ __forceinline__ void load_weight(const void *w, int f32, const Unit<TAIL> &u, float (&f)[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 1.0f;
    } else if (f32) {
        const float *p = reinterpret_cast<const float *>(static_cast<const char *>(w) + 4u * u.start);
        if (!TAIL || u.n >= 8) {
            const f32x4 a = *reinterpret_cast<const f32x4_row *>(p), b = *reinterpret_cast<const f32x4_row *>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = a[e];
                f[e + 4] = b[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < u.n ? p[e] : 0.0f;
        }
    } else {
        Wide<E>::widen(u.load(static_cast<const uint16_t *>(w)), f);
    }
}

// A sum over the L lanes of a row, or (L = 0) over the workgroup's waves.
// `part` holds one value per wave; a call's barrier separates its writes from
// its reads, and callers alternate between two of them.
template <int L>
__device__ __forceinline__ float sum_row(float v, float *part) {
    if constexpr (L > 0) {
        return sum_lanes<L>(v);
    } else {
        v = sum_lanes<kWave>(v);
        const int waves = (blockDim.x + kWave - 1) / kWave;
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
        __syncthreads();
        const int lane = threadIdx.x % kNormMaxWaves;
        return sum_lanes<kNormMaxWaves>(lane < waves ? part[lane] : 0.0f);
    }
}

template <int L>
__device__ __forceinline__ uint32_t max_row(uint32_t v, uint32_t *part) {
    if constexpr (L > 0) {
        return max_lanes<L>(v);
    } else {
        v = max_lanes<kWave>(v);
        const int waves = (blockDim.x + kWave - 1) / kWave;
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
        __syncthreads();
        const int lane = threadIdx.x % kNormMaxWaves;
        return max_lanes<kNormMaxWaves>(lane < waves ? part[lane] : 0u);
    }
}

__device__ __forceinline__ uint32_t max_of_group(uint32_t v, int lanes) {
    if (lanes == 16) return max_lanes<16>(v);
    if (lanes == 8) return max_lanes<8>(v);
    return max_lanes<4>(v);
}

// One row per workgroup (L = 0), or one row per L lanes of a workgroup.  Bound
// by HBM: 2048 x 8192 of eight contributions and a residual 60 us, 6.1 TB/s;
// 4999 x 5120 with both outputs 41.6 us, 5.5 TB/s.
// Thread t of a row holds units t, t + threads, .. (U of them) from the fold's
// loads to the stores, so every input byte is read once.  B operands are loaded
// at once: few, because registers held for loads keep waves off the compute
// unit (2048 x 8192 of one contribution with B = 9, 4 and 3: 26.7, 24.1 and
// 23.6 us; of eight 61.6, 60.6 and 60.7), unless there are too few rows for
// many waves anyway (kSpreadGroups).
template <class E, int U, int L, bool TAIL, bool NT, int B>
__global__ __launch_bounds__(kNormMaxThreads) void norm_rows(NormArgs a) {
    __shared__ float sums[kNormMaxWaves];
    __shared__ uint32_t maxs[kNormMaxWaves];
    const int threads = L > 0 ? L : static_cast<int>(blockDim.x);
    const int t = L > 0 ? static_cast<int>(threadIdx.x) % L : static_cast<int>(threadIdx.x);
    const size_t row = L > 0 ? static_cast<size_t>(blockIdx.x) * (blockDim.x / L) + threadIdx.x / (L > 0 ? L : 1)
                             : static_cast<size_t>(blockIdx.x);
    const int hidden = a.hidden;
    const int units = (hidden + 7) / 8;
    const bool there = L == 0 || row < a.rows;

    u32x4 h[U];
#pragma unroll
    for (int u = 0; u < U; ++u) h[u] = u32x4{0, 0, 0, 0};
    for (int g0 = 0; g0 < a.n; g0 += B) {
        u32x4 x[B][U];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int g = g0 + b;
            if (g < a.n) {
                const uint16_t *p = a.in[g] + row * (g == a.n - 1 ? a.last_stride : a.in_stride);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = t + u * threads;
                    x[b][u] = u32x4{0, 0, 0, 0};
                    if (there && i < units) x[b][u] = Unit<TAIL>(i, hidden).template load<NT>(p);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (g0 + b < a.n) {
#pragma unroll
                for (int u = 0; u < U; ++u) h[u] = (g0 + b == 0) ? x[b][u] : E::add8(h[u], x[b][u]);
            }
        }
    }

    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[8];
        Wide<E>::widen(h[u], f);
        const Unit<TAIL> at(t + u * threads, hidden);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = at.own(e) ? fmaf(f[e], f[e], sum) : sum;
    }
    float w[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = t + u * threads;
        if (i < units) load_weight<E>(a.weight, a.weight_f32, Unit<TAIL>(i, hidden), w[u]);
    }
    sum = sum_row<L>(sum, sums);
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(hidden) + a.eps);
    if (there && t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;

    float y[U][8];
    uint32_t top[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = t + u * threads;
        top[u] = 0;
        if (i >= units) continue;
        const Unit<TAIL> at(i, hidden);
        Wide<E>::widen(h[u], y[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[u][e] = y[u][e] * rstd * w[u][e];
            // magnitudes compared as integers, so that a NaN is the largest
            if (at.own(e)) {
                const uint32_t m = __builtin_bit_cast(uint32_t, y[u][e]) & 0x7FFFFFFFu;
                top[u] = top[u] > m ? top[u] : m;
            }
        }
        if (!there) continue;
        if (a.h != nullptr) at.template store<NT>(a.h + row * a.h_stride, h[u]);
        if (a.out != nullptr) at.template store<NT>(a.out + row * a.out_stride, Wide<E>::narrow(y[u]));
    }
    if (a.codes == nullptr) return;

    if (a.group_lanes == 0) {
        uint32_t m = top[0];
#pragma unroll
        for (int u = 1; u < U; ++u) m = m > top[u] ? m : top[u];
        m = max_row<L>(m, maxs);
#pragma unroll
        for (int u = 0; u < U; ++u) top[u] = m;
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) top[u] = max_of_group(top[u], a.group_lanes);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = t + u * threads;
        if (!there || i >= units) continue;
        const float m = __builtin_bit_cast(float, top[u]);
        const float scale = m < kE4m3Max * kMinScale ? kMinScale : m / kE4m3Max;   // NaN stays NaN
        if (a.group_lanes == 0 ? i == 0 : i % a.group_lanes == 0)
            a.scales[row * a.scales_stride + (a.group_lanes == 0 ? 0 : i / a.group_lanes)] = scale;
        // y / scale, rounded once, with one reciprocal for the group.  The product
        // with it is up to 1.5 units in the last place off, which moves quotients
        // half way between two codes.  A step by the remainder brings it within
        // one unit, and from there the next gives the division's own result
        // (Markstein 1990: a quotient within a unit, the reciprocal to nearest, an
        // exact remainder; the negated one keeps the sign of a zero).  Remainders
        // are exact for scales from 2^-90 on where a quotient is 2^-11 or more,
        // and smaller ones have the code 0; smaller scales are lifted.  What is
        // finite over an infinite scale is 0.  (16384 x 4096 of one contribution and
        // a residual 78.8 us, 84.0 with divisions, 77.6 with the bare product.)
        float divisor = scale;
        if (scale < 0x1p-90f) {
            divisor *= 0x1p60f;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[u][e] *= 0x1p60f;
        }
        const float inv = 1.0f / divisor;
        divisor = divisor == INFINITY ? 0.0f : divisor;
        const auto over = [&](float v) {
            float r = v * inv;
            r = fmaf(-fmaf(r, divisor, -v), inv, r);
            return fmaf(-fmaf(r, divisor, -v), inv, r);
        };
        u32x2 c;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(over(y[u][4 * q]), over(y[u][4 * q + 1]), 0, false);
            v = __builtin_amdgcn_cvt_pk_fp8_f32(over(y[u][4 * q + 2]), over(y[u][4 * q + 3]), v, true);
            c[q] = static_cast<uint32_t>(v);
        }
        // a last unit's shared values may have another group's scale: its own only
        const Unit<TAIL> at(i, hidden);
        uint8_t *p = a.codes + row * a.codes_stride + at.start;
        if (!TAIL || (hidden >= 8 && at.skip == 0)) {
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

struct NormGradArgs {
    const uint16_t *dy, *h, *dres;
    const float *rstd;
    const void *weight;
    uint16_t *dx;
    float *part;                     // one row of `hidden` sums per workgroup; null: not wanted
    size_t rows;
    size_t dy_stride, h_stride, dres_stride, dx_stride;
    int hidden;
    int weight_f32;
    uint32_t row_groups;             // workgroups for rows; the others sum columns
    float *dweight;                  // of these others
};

// Few rows: dweight = sum over the rows of dy * h * rstd without partial sums
// in memory.  A workgroup takes the columns of kColumnLanes units, its groups
// of so many lanes every so many rows, and the groups' sums are added in order.
// It reads dy and h once more, from the caches.  (In a graph, 4, 8 and 16
// lanes: 256 x 1024 4.2, 5.6 and 8.5 us, 256 x 8192 8.4, 7.4 and 8.5, 1 x 4096
// 3.8, 3.0 and 2.7.)
constexpr int kColumnLanes = 8;
constexpr int kColumns = 8 * kColumnLanes;

template <class E, bool TAIL>
__device__ __forceinline__ void sum_few_rows(const NormGradArgs &a) {
    extern __shared__ float cols[];                 // [groups][kColumns]
    const int groups = blockDim.x / kColumnLanes, group = threadIdx.x / kColumnLanes;
    const int lane = threadIdx.x % kColumnLanes, first = static_cast<int>(blockIdx.x - a.row_groups) * kColumnLanes;
    const Unit<TAIL> at(first + lane, a.hidden);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    if (8 * (first + lane) < a.hidden) {
#pragma unroll 4
        for (size_t row = group; row < a.rows; row += groups) {
            float dy[8], h[8];
            Wide<E>::widen(at.load(a.dy + row * a.dy_stride), dy);
            Wide<E>::widen(at.load(a.h + row * a.h_stride), h);
            const float rstd = a.rstd[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(dy[e], h[e] * rstd, acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) cols[group * kColumns + lane * 8 + e] = acc[e];
    __syncthreads();
    for (int c = threadIdx.x; c < kColumns; c += blockDim.x) {
        float s = cols[c];
        for (int g = 1; g < groups; ++g) s += cols[g * kColumns + c];
        // (a last unit lies before its place in the workgroup's columns)
        const Unit<TAIL> u(first + c / 8, a.hidden);
        if (8 * (first + c / 8) < a.hidden && u.own(c % 8)) a.dweight[u.start + c % 8] = s;
    }
}

// dx = rstd * (g - u * mean(g u)) + dres with g = dy * weight, u = h * rstd,
// and this workgroup's sum over its rows of dy * u.  Rows are dealt out to the
// workgroups (L = 0) or to groups of L lanes in turn; a thread keeps its
// columns' sums in registers from its first row to its last.  Bound by HBM:
// 2048 x 8192 with dres and dweight 31 us, of which 4 are sum_columns.  (Loading
// a row ahead was no faster: 33.9 against 33.0 us at the time.)  Rows of more than
// 16384 values (U = 4) are read twice: 8192 x 20000 382 us, 8192 x 16384 181.
// FEW: further workgroups sum the columns (in kernels of their own, since that
// takes registers).
template <class E, int U, int L, bool TAIL, bool NT, bool FEW>
__global__ __launch_bounds__(kNormMaxThreads) void norm_grad_rows(NormGradArgs a) {
    if constexpr (FEW) {
        if (blockIdx.x >= a.row_groups) {
            sum_few_rows<E, TAIL>(a);
            return;
        }
    }
    __shared__ float sums[2][kNormMaxWaves];
    const int threads = L > 0 ? L : static_cast<int>(blockDim.x);
    const int t = L > 0 ? static_cast<int>(threadIdx.x) % L : static_cast<int>(threadIdx.x);
    const int per = L > 0 ? static_cast<int>(blockDim.x) / (L > 0 ? L : 1) : 1;
    const size_t step = static_cast<size_t>(a.row_groups) * per;
    const int hidden = a.hidden;
    const int units = (hidden + 7) / 8;

    float acc[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[u][e] = 0.0f;

    // Up to two units per thread the row stays in registers between its two
    // uses, and the weights from row to row; four would spill.
    constexpr bool kKeep = U <= 2;
    float kept[kKeep ? U : 1][8];
    if constexpr (kKeep) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int e = 0; e < 8; ++e) kept[u][e] = 0.0f;
            if (t + u * threads < units)
                load_weight<E>(a.weight, a.weight_f32, Unit<TAIL>(t + u * threads, hidden), kept[u]);
        }
    }

    int turn = 0;
    for (size_t row0 = static_cast<size_t>(blockIdx.x) * per; row0 < a.rows; row0 += step, turn ^= 1) {
        const size_t row = row0 + (L > 0 ? threadIdx.x / (L > 0 ? L : 1) : 0);
        const bool there = L == 0 || row < a.rows;
        const float rstd = there ? a.rstd[row] : 0.0f;
        u32x4 d[U], h[U], r[U];
        auto load = [&](int u) {
            const int i = t + u * threads;
            d[u] = h[u] = r[u] = u32x4{0, 0, 0, 0};
            if (there && i < units) {
                const Unit<TAIL> at(i, hidden);
                d[u] = at.template load<NT>(a.dy + row * a.dy_stride);
                h[u] = at.template load<NT>(a.h + row * a.h_stride);
                if (a.dres != nullptr) r[u] = at.template load<NT>(a.dres + row * a.dres_stride);
            }
        };
        if constexpr (kKeep) {
#pragma unroll
            for (int u = 0; u < U; ++u) load(u);
        }
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = t + u * threads;
            Unit<TAIL> at(i, hidden);
            // (hidden from the compiler, which would keep every unit's masks)
            if constexpr (!kKeep) asm volatile("" : "+v"(at.skip));
            float dy[8], unit[8], w[8];
            if constexpr (!kKeep) load(u);
            Wide<E>::widen(d[u], dy);
            Wide<E>::widen(h[u], unit);
            if constexpr (kKeep) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = kept[u][e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 0.0f;
                if (i < units) load_weight<E>(a.weight, a.weight_f32, Unit<TAIL>(i, hidden), w);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                unit[e] *= rstd;
                acc[u][e] = fmaf(dy[e], unit[e], acc[u][e]);
                sum = at.own(e) ? fmaf(dy[e] * w[e], unit[e], sum) : sum;
            }
            if constexpr (!kKeep) {
                // one unit at a time: the empty statement stops the compiler
                // from loading all of them first, which spills
#pragma unroll
                for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(acc[u][e]));
                asm volatile("" : "+v"(sum)::"memory");
            }
        }
        const float mean = sum_row<L>(sum, sums[turn]) / static_cast<float>(hidden);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = t + u * threads;
            if (!there || i >= units) continue;
            float dy[8], unit[8], w[8], f[8];
            if constexpr (!kKeep) {
                load(u);   // again (below the streaming limit from the caches)
            }
            Wide<E>::widen(d[u], dy);
            Wide<E>::widen(h[u], unit);
            Wide<E>::widen(r[u], f);
            if constexpr (kKeep) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = kept[u][e];
            } else {
                load_weight<E>(a.weight, a.weight_f32, Unit<TAIL>(i, hidden), w);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += rstd * (dy[e] * w[e] - unit[e] * rstd * mean);
            // (rows that are read twice may be overwritten between the reads
            // of a shared value)
            const Unit<TAIL> at(i, hidden);
            if constexpr (kKeep)
                at.template store<NT>(a.dx + row * a.dx_stride, Wide<E>::narrow(f));
            else
                at.template store_own<NT>(a.dx + row * a.dx_stride, Wide<E>::narrow(f));
            if constexpr (!kKeep) asm volatile("" ::: "memory");
        }
    }
    if (a.part == nullptr) return;
    float *part = a.part + static_cast<size_t>(blockIdx.x) * hidden;
    if constexpr (L > 0) {
        // the row groups of the workgroup, added in order
        __shared__ float cols[4 * kWave * 8];       // 256 threads at most (launch)
        const Unit<TAIL> at(t, hidden);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (t < units && at.own(e)) cols[threadIdx.x / L * (L * 8) + at.start + e] = acc[0][e];
        __syncthreads();
        for (int c = threadIdx.x; c < hidden; c += blockDim.x) {
            float s = 0.0f;
            for (int k = 0; k < per; ++k) s += cols[k * (L * 8) + c];
            part[c] = s;
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = t + u * threads;
            if (i >= units) continue;
            const Unit<TAIL> at(i, hidden);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at.own(e)) part[at.start + e] = acc[u][e];
        }
    }
}

// out[c] = sum over p of part[p][c], in a fixed order: a workgroup takes C
// columns, its groups of C lanes every so many rows, and the groups' sums are
// added in order.  Fewer columns to a workgroup make more workgroups of short
// rows.
constexpr int kColumnThreads = 1024;

template <int C>
__global__ __launch_bounds__(kColumnThreads) void sum_columns(const float *part, size_t parts, int hidden, float *out) {
    constexpr int kGroups = kColumnThreads / C;
    __shared__ float sums[kGroups][C];
    const int c = static_cast<int>(blockIdx.x) * C + threadIdx.x % C;
    const int group = threadIdx.x / C;
    float s = 0.0f;
    if (c < hidden) {
#pragma unroll 8
        for (size_t p = group; p < parts; p += kGroups) s += part[p * hidden + c];
    }
    sums[group][threadIdx.x % C] = s;
    __syncthreads();
    if (group == 0 && c < hidden) {
        s = sums[0][threadIdx.x];
        for (int k = 1; k < kGroups; ++k) s += sums[k][threadIdx.x];
        out[c] = s;
    }
}

namespace {

constexpr int kRowGroupThreads = 256;

// How a row of `hidden` values is laid over threads.
struct RowShape {
    int lanes;     // lanes per row; 0 = a workgroup per row
    int units;     // units of 8 values per thread
    int threads;   // of a workgroup
};

RowShape row_shape(int hidden, bool spread = false) {
    const int units = (hidden + 7) / 8;
    if (units <= 16) return {16, 1, kRowGroupThreads};
    if (units <= 32) return {32, 1, kRowGroupThreads};
    if (units <= 64) return {64, 1, kRowGroupThreads};
    const int per = units <= (spread ? 1024 : 512) ? 1 : units <= 2048 ? 2 : 4;
    const int threads = ((units + per - 1) / per + kWave - 1) / kWave * kWave;
    return {0, per, threads};
}

// Few workgroups with many operands wait for their loads: nine operands at
// once, and of long rows one unit per thread, twice the threads.  (In a graph,
// with binary16 output alone, 64 x 6144 of eight contributions 5.6 us with two
// units per thread, 5.0 with one and four operands at once, 4.1 with nine, and 5.4
// from bfloat16 to e4m3 with scales of 128; 2048 x 8192 of eight 61.6 with
// two units and 67.8 with one; 8192 x 64 of sixteen 8.4 us with four operands at
// once, 6.5 with nine, 32768 x 64 15.1 either way.)
constexpr size_t kSpreadGroups = 512;
constexpr int kSpreadOperands = 5;

// A call that moves this many bytes or more passes the caches by
// (non-temporal loads and stores).  Measured cached and streamed over buffers
// that the caches no longer hold (three sets in turn): the fold of 8
// contributions of 2048 x 8192 (369 MB) 71.3 and 59.8 us, one of 4999 x 5120
// with both outputs (230 MB) 46.2 and 40.8, the gradient of 8192 x 4096 (268
// MB) 54.8 and 50.1, of 1024 x 8192 (67 MB) 16.8 and 20.4.  Between copies that
// write its contributions and read its output, on one set: 2048 x 8192 of one
// (134 MB) 42.3 and 47.0 in all, 32768 x 1024 of one (268 MB) 89.7 and 88.0,
// 2048 x 8192 of eight 191 and 179; smaller ones keep what the caches hold
// (1000 x 5121 of eight 60.9 and 72.1), though alone they would be faster
// streamed (33.8 and 28.8).
constexpr size_t kStreamBytes = size_t(1) << 27;

// How a call's kernel differs beside its row's layout.
enum Mode {
    kCached,
    kStreamed,
    kSmall        // norm: spread (kSpreadGroups); gradient: few rows
};

template <template <class, int, int, bool, Mode> class K, class E, class A>
hipError_t launch_rows(const RowShape &s, bool tail, Mode mode, size_t grid, size_t lds, hipStream_t stream,
                       const A &args) {
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(s.threads), lds, stream, args);
        return hipGetLastError();
    };
#define HR_MODE(U, L, TAIL)                                        \
    (mode == kCached     ? K<E, U, L, TAIL, kCached>::kernel       \
     : mode == kStreamed ? K<E, U, L, TAIL, kStreamed>::kernel     \
                         : K<E, U, L, TAIL, kSmall>::kernel)
#define HR_VARIANT(U, L) (tail ? HR_MODE(U, L, true) : HR_MODE(U, L, false))
    switch (s.lanes) {
        case 16: return go(HR_VARIANT(1, 16));
        case 32: return go(HR_VARIANT(1, 32));
        case 64: return go(HR_VARIANT(1, 64));
    }
    if (s.units == 1) return go(HR_VARIANT(1, 0));
    if (s.units == 2) return go(HR_VARIANT(2, 0));
    return go(HR_VARIANT(4, 0));
#undef HR_VARIANT
#undef HR_MODE
}

template <class E, int U, int L, bool TAIL, Mode M>
struct NormKernel {
    static constexpr int kOperandsAtOnce = U == 4 ? 2 : U == 1 && M == kSmall ? 9 : 4;
    static constexpr auto kernel = norm_rows<E, U, L, TAIL, M == kStreamed, kOperandsAtOnce>;
};

template <class E, int U, int L, bool TAIL, Mode M>
struct NormGradKernel {
    static constexpr auto kernel = norm_grad_rows<E, U, L, TAIL, M == kStreamed, M == kSmall>;
};

constexpr size_t kMaxRows = 0x7FFFFFFF;

size_t groups_of(size_t rows, const RowShape &s) {
    const size_t per = s.lanes > 0 ? s.threads / s.lanes : 1;
    return (rows + per - 1) / per;
}

// Workgroups of the gradient, hence partial sums of dweight.  Up to four on a
// compute unit and 16 waves (8 where a workgroup takes several rows at once),
// but with eight rows or more to each, so that the partial sums stay small
// beside the rows: one on a compute unit at least, and where rows are short two
// while each has two rows.  (16384 x 1024 with 512, 1024 and 2048 workgroups:
// 40, 30 and 34 us; 4097 x 5120 with 256 and 512: 41 and 35; 2048 x 8192 with
// 256, 512 and 1024: 31, 33 and 36; 2048 x 2048 with 256, 512 and 1024: 14.1,
// 12.2 and 14.3; 759 x 4096 with 256 and 380: 10.8 and 13.3.)
constexpr int kShortRow = 2048;

size_t grad_groups(size_t rows, int hidden, int cus) {
    const RowShape s = row_shape(hidden);
    const size_t groups = groups_of(rows, s), n = static_cast<size_t>(cus);
    const int fit = (s.lanes > 0 ? 8 : 16) * kWave / s.threads;
    const size_t most = n * (fit < 1 ? 1 : fit < 4 ? fit : 4);
    const size_t two = groups / 2 < 2 * n ? groups / 2 : 2 * n;
    const size_t least = hidden <= kShortRow && two > n ? two : n;
    const size_t deep = groups / 8 > least ? groups / 8 : least;
    const size_t cap = deep < most ? deep : most;
    return groups < cap ? groups : cap;
}

// The largest number of compute units a device of this kind has; the workspace
// is sized without asking a device.
constexpr int kMaxCus = 256;

bool any_overlap(const Region *outs, int no, const Region *ins, int ni, unsigned in_place) {
    for (int o = 0; o < no; ++o) {
        for (int i = 0; i < ni; ++i)
            if (regions_overlap(outs[o], ins[i]) && !((in_place >> o & 1) && regions_same(outs[o], ins[i]))) return true;
        for (int p = 0; p < o; ++p)
            if (regions_overlap(outs[o], outs[p])) return true;
    }
    return false;
}

template <class E>
hr_status norm_impl(const hr_rmsnorm_args *q, hr_stream_t stream) {
    if (q == nullptr || q->G < 1 || q->G > HR_MAX_G || q->hidden == 0 || !(q->eps >= 0.0f)) return HR_ERR_INVALID_ARG;
    if (q->group != 0 && q->group != 32 && q->group != 64 && q->group != 128) return HR_ERR_INVALID_ARG;
    if (q->hidden > HR_RMSNORM_MAX_HIDDEN || q->rows > kMaxRows) return HR_ERR_TOO_LARGE;
    if (q->rows == 0) return HR_OK;
    const bool spread = groups_of(q->rows, row_shape(static_cast<int>(q->hidden), true)) <= kSpreadGroups &&
                        q->G + (q->residual != nullptr) >= kSpreadOperands;
    const RowShape s = row_shape(static_cast<int>(q->hidden), spread);
    if (groups_of(q->rows, s) > 0xFFFFFFFFu / s.threads) return HR_ERR_TOO_LARGE;   // work-items of a launch
    if (q->out == nullptr && q->residual_out == nullptr && q->codes == nullptr && q->rstd == nullptr)
        return HR_ERR_INVALID_ARG;
    if ((q->codes == nullptr) != (q->scales == nullptr)) return HR_ERR_INVALID_ARG;

    const size_t rows = q->rows, hidden = q->hidden;
    const size_t groups = q->group == 0 ? 1 : (hidden + q->group - 1) / q->group;
    NormArgs a{};
    a.in_stride = q->input_stride;
    a.last_stride = q->residual_stride;
    a.h_stride = q->residual_out_stride;
    a.out_stride = q->out_stride;
    a.codes_stride = q->codes_stride;
    a.scales_stride = q->scales_stride;
    if (!row_stride(rows, hidden, &a.in_stride, 2) || !row_stride(rows, hidden, &a.last_stride, 2) ||
        !row_stride(rows, hidden, &a.h_stride, 2) || !row_stride(rows, hidden, &a.out_stride, 2) ||
        !row_stride(rows, hidden, &a.codes_stride, 1) || !row_stride(rows, groups, &a.scales_stride, 4))
        return HR_ERR_INVALID_ARG;

    Region ins[kOperands];
    int ni = 0;
    for (int g = 0; g < q->G; ++g) {
        if (q->inputs[g] == nullptr) return HR_ERR_INVALID_ARG;
        if (!aligned(q->inputs[g], 2)) return HR_ERR_ALIGNMENT;
        a.in[g] = static_cast<const uint16_t *>(q->inputs[g]);
        ins[ni++] = Region{q->inputs[g], rows, hidden * 2, a.in_stride * 2};
    }
    a.n = q->G;
    if (q->residual != nullptr) {
        if (!aligned(q->residual, 2)) return HR_ERR_ALIGNMENT;
        a.in[a.n++] = static_cast<const uint16_t *>(q->residual);
        ins[ni++] = Region{q->residual, rows, hidden * 2, a.last_stride * 2};
    } else {
        a.last_stride = a.in_stride;
    }
    if (!aligned(q->weight, q->weight_f32 ? 4 : 2)) return HR_ERR_ALIGNMENT;
    const Region weight = {q->weight, 1, hidden * (q->weight_f32 ? 4 : 2), 0};
    if (!aligned(q->residual_out, 2) || !aligned(q->out, 2) || !aligned(q->scales, 4) || !aligned(q->rstd, 4))
        return HR_ERR_ALIGNMENT;
    const Region outs[] = {{q->residual_out, rows, hidden * 2, a.h_stride * 2},
                           {q->out, rows, hidden * 2, a.out_stride * 2},
                           {q->codes, rows, hidden, a.codes_stride},
                           {q->scales, rows, groups * 4, a.scales_stride * 4},
                           {q->rstd, rows, 4, 4}};
    // a row is read whole before any of it is written, so the 16-bit outputs
    // may take an input's place
    if (any_overlap(outs, 5, ins, ni, 0x3) || any_overlap(outs, 5, &weight, 1, 0)) return HR_ERR_INVALID_ARG;

    a.weight = q->weight;
    a.weight_f32 = q->weight_f32 != 0;
    a.h = static_cast<uint16_t *>(q->residual_out);
    a.out = static_cast<uint16_t *>(q->out);
    a.codes = static_cast<uint8_t *>(q->codes);
    a.scales = q->scales;
    a.rstd = q->rstd;
    a.rows = rows;
    a.hidden = static_cast<int>(hidden);
    a.group_lanes = q->group / 8;
    a.eps = q->eps;

    const size_t arrays = a.n + (a.h != nullptr) + (a.out != nullptr) + (a.codes != nullptr);
    const Mode mode = rows * hidden * 2 * arrays >= kStreamBytes ? kStreamed : spread ? kSmall : kCached;
    const hipError_t e = launch_rows<NormKernel, E>(s, hidden % 8 != 0, mode, groups_of(rows, s), 0,
                                                    reinterpret_cast<hipStream_t>(stream), a);
    return e == hipSuccess ? HR_OK : HR_ERR_HIP;
}

template <class E>
hr_status norm_grad_impl(const hr_rmsnorm_grad_args *q, hr_stream_t stream) {
    if (q == nullptr || q->hidden == 0) return HR_ERR_INVALID_ARG;
    if (q->hidden > HR_RMSNORM_MAX_HIDDEN || q->rows > kMaxRows) return HR_ERR_TOO_LARGE;
    const size_t rows = q->rows, hidden = q->hidden;
    if (rows == 0 && q->dweight == nullptr) return HR_OK;
    if (rows > 0 && (q->dy == nullptr || q->h == nullptr || q->rstd == nullptr || q->dx == nullptr))
        return HR_ERR_INVALID_ARG;
    NormGradArgs a{};
    a.dy_stride = q->dy_stride;
    a.h_stride = q->h_stride;
    a.dres_stride = q->dresidual_stride;
    a.dx_stride = q->dx_stride;
    if (!row_stride(rows, hidden, &a.dy_stride, 2) || !row_stride(rows, hidden, &a.h_stride, 2) ||
        !row_stride(rows, hidden, &a.dres_stride, 2) || !row_stride(rows, hidden, &a.dx_stride, 2))
        return HR_ERR_INVALID_ARG;
    if (!aligned(q->dy, 2) || !aligned(q->h, 2) || !aligned(q->dresidual, 2) || !aligned(q->dx, 2) ||
        !aligned(q->weight, q->weight_f32 ? 4 : 2) || !aligned(q->rstd, 4) || !aligned(q->dweight, 4) ||
        !aligned(q->workspace, 4))
        return HR_ERR_ALIGNMENT;

    int dev = 0, cus = 0;
    const Region dx = {q->dx, rows, hidden * 2, a.dx_stride * 2};
    const Region dy = {q->dy, rows, hidden * 2, a.dy_stride * 2}, h = {q->h, rows, hidden * 2, a.h_stride * 2};
    const bool few = q->dweight != nullptr && rows > 0 && rows <= HR_RMSNORM_GRAD_FEW_ROWS &&
                     !regions_overlap(dx, dy) && !regions_overlap(dx, h);
    const size_t need = few ? 0 : hr_rmsnorm_grad_workspace(rows, hidden);
    if (q->dweight != nullptr && need > 0 && (q->workspace == nullptr || q->workspace_bytes < need))
        return HR_ERR_INVALID_ARG;
    const size_t used = q->dweight != nullptr ? need : 0;
    const Region ins[] = {dy, h, {q->dresidual, rows, hidden * 2, a.dres_stride * 2}};
    const Region others[] = {{q->weight, 1, hidden * (q->weight_f32 ? 4 : 2), 0}, {q->rstd, rows, 4, 4}};
    const Region outs[] = {dx,
                           {q->dweight, 1, hidden * 4, 0},
                           {q->workspace, 1, used, 0}};
    if (any_overlap(outs, 3, ins, 3, 0x1) || any_overlap(outs, 3, others, 2, 0)) return HR_ERR_INVALID_ARG;
    if (stream_device(stream, &dev) != hipSuccess) return HR_ERR_HIP;
    if (device_cu_count(dev, &cus) != hipSuccess) return HR_ERR_HIP;
    if (cus > kMaxCus) cus = kMaxCus;
    const hipStream_t st = reinterpret_cast<hipStream_t>(stream);

    a.dy = static_cast<const uint16_t *>(q->dy);
    a.h = static_cast<const uint16_t *>(q->h);
    a.dres = static_cast<const uint16_t *>(q->dresidual);
    a.rstd = q->rstd;
    a.weight = q->weight;
    a.weight_f32 = q->weight_f32 != 0;
    a.dx = static_cast<uint16_t *>(q->dx);
    a.rows = rows;
    a.hidden = static_cast<int>(hidden);
    const RowShape s = row_shape(a.hidden);
    const bool tail = hidden % 8 != 0;
    if (few) {
        const size_t groups = groups_of(rows, s), columns = (hidden + kColumns - 1) / kColumns;
        a.row_groups = static_cast<uint32_t>(groups);
        a.dweight = q->dweight;
        const hipError_t e = launch_rows<NormGradKernel, E>(s, tail, kSmall, groups + columns,
                                                            s.threads / kColumnLanes * kColumns * sizeof(float), st, a);
        return e == hipSuccess ? HR_OK : HR_ERR_HIP;
    }
    const size_t parts = grad_groups(rows, a.hidden, cus);
    // a single workgroup's sums are the result
    float *part = parts == 1 ? q->dweight : static_cast<float *>(q->workspace);
    a.part = q->dweight != nullptr ? part : nullptr;
    a.row_groups = static_cast<uint32_t>(parts);
    if (rows > 0) {
        const size_t arrays = 3 + (a.dres != nullptr);
        const Mode mode = rows * hidden * 2 * arrays >= kStreamBytes ? kStreamed : kCached;
        const hipError_t e = launch_rows<NormGradKernel, E>(s, tail, mode, parts, 0, st, a);
        if (e != hipSuccess) return HR_ERR_HIP;
    }
    if (q->dweight != nullptr && parts != 1) {
        const int columns = hidden >= 4096 ? 64 : 16;
        const dim3 grid(static_cast<unsigned>((hidden + columns - 1) / columns));
        const float *sums = static_cast<const float *>(q->workspace);
        if (columns == 64)
            hipLaunchKernelGGL(sum_columns<64>, grid, dim3(kColumnThreads), 0, st, sums, parts, a.hidden, q->dweight);
        else
            hipLaunchKernelGGL(sum_columns<16>, grid, dim3(kColumnThreads), 0, st, sums, parts, a.hidden, q->dweight);
        if (hipGetLastError() != hipSuccess) return HR_ERR_HIP;
    }
    return HR_OK;
}

}  // namespace

}  // namespace hr

using namespace hr;

extern "C" HR_API hr_status hr_reduce_rmsnorm_f16(const hr_rmsnorm_args *args, hr_stream_t stream) {
    return norm_impl<F16>(args, stream);
}

extern "C" HR_API hr_status hr_reduce_rmsnorm_bf16(const hr_rmsnorm_args *args, hr_stream_t stream) {
    return norm_impl<BF16>(args, stream);
}

extern "C" HR_API hr_status hr_rmsnorm_grad_f16(const hr_rmsnorm_grad_args *args, hr_stream_t stream) {
    return norm_grad_impl<F16>(args, stream);
}

extern "C" HR_API hr_status hr_rmsnorm_grad_bf16(const hr_rmsnorm_grad_args *args, hr_stream_t stream) {
    return norm_grad_impl<BF16>(args, stream);
}

extern "C" HR_API size_t hr_rmsnorm_grad_workspace(size_t rows, size_t hidden) {
    if (rows > kMaxRows || hidden == 0 || hidden > HR_RMSNORM_MAX_HIDDEN) return 0;
    const size_t parts = grad_groups(rows, static_cast<int>(hidden), kMaxCus);
    return parts > 1 ? parts * hidden * sizeof(float) : 0;
}
