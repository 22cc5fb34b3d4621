// experts.hip -- tokens sorted by expert and back.
//
//   hr_experts_sort          where each (token, pick) goes: a stable counting
//                            sort of the picks by expert
//   hr_experts_gather        rows copied to their sorted places
//   hr_experts_combine       y[t] = sum_j weights[t][j] * z[pos[t][j]] (+ addend)
//   hr_experts_combine_grad  dz[pos[t][j]] = weights[t][j] * dy[t],
//                            dweights[t][j] = <dy[t], z[pos[t][j]]>
//
// (The gradient of the gather is the combine without weights.)  Apart from
// the sort, every kernel moves rows once and is bound by HBM: a workgroup (or
// a part of it, for short rows) takes a token, so the token's own row is read
// or written once and its k expert rows are all in flight together.
#include "rows.h"

#include <type_traits>

namespace hr {

constexpr int kExpertThreads = 256;
constexpr int kMaxSortThreads = 1024;

// ------------------------------------------------------------------ the sort

struct SortArgs {
    const int32_t *ids;
    int32_t *offsets, *order, *pos;
    int32_t *counts;         // [blocks][experts]
    uint32_t slots, rows;
    uint32_t chunk;          // slots per workgroup
    int first, experts, pad;
    int bits;                // of an expert's number, `experts` (none) included
    int blocks;
};

// The experts of N slots s, s + step, .. below end, their ids loaded together,
// counted from `first`: `experts` for a slot that goes nowhere, -1 from end on.
template <int N>
__device__ __forceinline__ void load_experts(const SortArgs &a, uint32_t s, uint32_t step, uint32_t end,
                                             int (&e)[N]) {
    int id[N];
#pragma unroll
    for (int i = 0; i < N; ++i) id[i] = s + i * step < end ? a.ids[s + i * step] : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t x = static_cast<uint32_t>(id[i]) - static_cast<uint32_t>(a.first);
        const bool here = id[i] >= a.first && x < static_cast<uint32_t>(a.experts);
        e[i] = s + i * step < end ? here ? static_cast<int>(x) : a.experts : -1;
    }
}

// Lanes of the wave that hold the same number: those that agree in every bit.
__device__ __forceinline__ uint64_t same_lanes(int e, int bits) {
    uint32_t lo = ~0u, hi = ~0u;
    for (int b = 0; b < bits; ++b) {
        const uint32_t mine = static_cast<uint32_t>(__builtin_amdgcn_sbfe(e, b, 1));      // all ones or zeros
        const uint64_t ones = __builtin_amdgcn_ballot_w64(mine != 0);
        lo &= ~(static_cast<uint32_t>(ones) ^ mine);
        hi &= ~(static_cast<uint32_t>(ones >> 32) ^ mine);
    }
    return lo | static_cast<uint64_t>(hi) << 32;
}

// counts[e] += a lane's slots of expert e.
template <int N>
__device__ __forceinline__ void count_experts(const SortArgs &a, const int (&e)[N], int *counts) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        // whole numbers: the order does not matter
        if (static_cast<uint32_t>(e[i]) < static_cast<uint32_t>(a.experts)) atomicAdd(&counts[e[i]], 1);
}

// The share of a workgroup's slots [begin, end) that a wave takes, in order.
__device__ __forceinline__ void wave_share(uint32_t begin, uint32_t end, int wave, int waves, uint32_t *b, uint32_t *e) {
    const uint32_t per = ((end - begin + waves - 1) / waves + kWave - 1) / kWave * kWave;
    *b = begin + wave * per < end ? begin + wave * per : end;
    *e = *b + per < end ? *b + per : end;
}

// A wave's slots of [begin, end) counted, N of a lane at a time; `e` keeps the
// last of them.
template <int N>
__device__ __forceinline__ void count_share(const SortArgs &a, uint32_t begin, uint32_t end, int *counts,
                                            int (&e)[N]) {
    for (uint32_t s = begin; s < end; s += kWave * N) {
        load_experts(a, s + threadIdx.x % kWave, kWave, end, e);
        count_experts(a, e, counts);
    }
}

// The wave's slots to their places: next[x] is the place of the next slot of
// expert x in this wave's share.  `e` is from count_share: the ids of a share of
// up to N slots a lane are not loaded again.
template <int N>
__device__ __forceinline__ void place_share(const SortArgs &a, uint32_t begin, uint32_t end, int *next,
                                            int (&e)[N]) {
    const uint32_t lane = threadIdx.x % kWave;
    for (uint32_t s0 = begin; s0 < end; s0 += kWave * N) {
        if (end - begin > kWave * N) load_experts(a, s0 + lane, kWave, end, e);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (s0 + i * kWave >= end) break;
            const int x = e[i];
            const bool goes = static_cast<uint32_t>(x) < static_cast<uint32_t>(a.experts);
            const uint64_t mask = same_lanes(x, a.bits);
            const int rank = __builtin_popcountll(mask & ((1ull << lane) - 1));
            int place = -1;
            if (goes) place = next[x] + rank;
            // every lane has read its expert's place before one of them moves it
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (goes && rank == 0) next[x] = place + __builtin_popcountll(mask);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (x >= 0) {
                const uint32_t s = s0 + i * kWave + lane;
                a.pos[s] = place;
                if (place >= 0) a.order[place] = static_cast<int32_t>(s);
            }
        }
    }
}

// Inclusive sums of v over the workgroup's threads, and their total; `tmp`
// holds a value per wave.  Every thread of the workgroup calls it, with a
// barrier between two calls on the same `tmp`.
__device__ __forceinline__ int scan_threads(int v, int *tmp, int *total) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int before = __shfl_up(v, d);
        v += lane >= d ? before : 0;
    }
    if (lane == kWave - 1) tmp[wave] = v;
    __syncthreads();
    int sum = 0;
    for (int w = 0; w < waves; w += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = tmp[w + i];
            v += w + i < wave ? n : 0;
            sum += n;
        }
    }
    *total = sum;
    return v;
}

// counts[w][x] of every wave w, to the place of expert x's first slot in that
// wave's share, from `at` on.  (Four waves at a time, as LDS takes its time.)
__device__ __forceinline__ void counts_to_places(int *counts, int experts, int x, int waves, int at) {
    for (int w = 0; w < waves; w += 4) {
        int n[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) n[i] = counts[(w + i) * experts + x];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            counts[(w + i) * experts + x] = at;
            at += n[i];
        }
    }
}

__device__ __forceinline__ int padded(int count, int pad) { return (count + pad - 1) / pad * pad; }

// order = -1 in the segments' padding, from their counts, and past the last
// segment; the experts and the tail are dealt out to the workgroups.  A lane
// looks at an expert, and the wave fills the segments that want it in turn.
__device__ __forceinline__ void fill_padding(const SortArgs &a, const int *offsets, const int *counts) {
    if (a.pad > 1) {
        const int waves = gridDim.x * (blockDim.x / kWave), lane = threadIdx.x % kWave;
        for (int e = (blockIdx.x * blockDim.x + threadIdx.x) / kWave; e < a.experts; e += kWave * waves) {
            const int x = e + lane * waves;
            const int from = x < a.experts ? offsets[x] + counts[x] : 0, to = x < a.experts ? offsets[x + 1] : 0;
            for (uint64_t m = __builtin_amdgcn_ballot_w64(from < to); m != 0; m &= m - 1) {
                const int l = __builtin_ctzll(m);
                const uint32_t begin = __builtin_amdgcn_readlane(from, l), end = __builtin_amdgcn_readlane(to, l);
                for (uint32_t p = begin + lane; p < end; p += kWave) a.order[p] = -1;
            }
        }
    }
    for (size_t p = static_cast<size_t>(offsets[a.experts]) + blockIdx.x * blockDim.x + threadIdx.x; p < a.rows;
         p += static_cast<size_t>(gridDim.x) * blockDim.x)
        a.order[p] = -1;
}

// Everything in one workgroup: 8 slots 3.0 us, 4096 slots of 128 experts 6.1,
// 8192 8.2, of which a launch is 1.6; the rest are the barriers and, per wave,
// 64 slots after another.  (Loading every 64 slots' ids when their turn comes,
// and again to place them, took 7.1 and 10.9.)  Dynamic LDS: [waves][experts]
// counts, then [experts + 1] offsets, [experts] totals and [waves] for the scan.
template <int N>
__global__ __launch_bounds__(kMaxSortThreads) void sort_once(SortArgs a) {
    extern __shared__ int lds[];
    const int waves = blockDim.x / kWave, wave = threadIdx.x / kWave;
    int *counts = lds, *offsets = counts + waves * a.experts, *totals = offsets + a.experts + 1,
        *tmp = totals + a.experts;
    for (int i = threadIdx.x; i < waves * a.experts; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    uint32_t b, e;
    wave_share(0, a.slots, wave, waves, &b, &e);
    int mine[N];
    count_share(a, b, e, counts + wave * a.experts, mine);
    __syncthreads();
    for (int e0 = 0, base = 0; e0 < a.experts; e0 += blockDim.x) {
        const int x = e0 + threadIdx.x;
        int sum = 0;
        if (x < a.experts)
            for (int w = 0; w < waves; w += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum += counts[(w + i) * a.experts + x];
        int all = 0;
        const int end = base + scan_threads(padded(sum, a.pad), tmp, &all);
        if (x < a.experts) {
            const int at = end - padded(sum, a.pad);
            totals[x] = sum;
            offsets[x] = at;
            offsets[x + 1] = end;      // the same value as its neighbour's own
            counts_to_places(counts, a.experts, x, waves, at);
        }
        base += all;
        __syncthreads();
    }
    for (int i = threadIdx.x; i <= a.experts; i += blockDim.x) a.offsets[i] = offsets[i];
    place_share(a, b, e, counts + wave * a.experts, mine);
    fill_padding(a, offsets, totals);
}

// The same over many workgroups: counts, then places.  Dynamic LDS: [experts].
template <int N>
__global__ __launch_bounds__(kMaxSortThreads) void sort_count(SortArgs a) {
    extern __shared__ int lds[];
    for (int i = threadIdx.x; i < a.experts; i += blockDim.x) lds[i] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * a.chunk;
    const uint32_t end = begin + a.chunk < a.slots ? begin + a.chunk : a.slots;
    for (uint32_t s = begin; s < end; s += N * blockDim.x) {
        int e[N];
        load_experts(a, s + threadIdx.x, blockDim.x, end, e);
        count_experts(a, e, lds);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.experts; i += blockDim.x) a.counts[blockIdx.x * a.experts + i] = lds[i];
}

// Every workgroup adds the counts of all of them up by itself: in a graph both
// kernels take 9.4 us for 65528 slots of 128 experts, 18.3 for 2^20 of 256.  (With
// a kernel of one workgroup between the two, 12.9 against 10.4 and 27.7 against
// 18.5 when these were measured.)
// Dynamic LDS: [waves][experts] counts, then [experts + 1] offsets, [experts]
// totals, [experts] firsts, [threads] sums and [waves].
template <int N>
__global__ __launch_bounds__(kMaxSortThreads) void sort_place(SortArgs a) {
    extern __shared__ int lds[];
    const int waves = blockDim.x / kWave, wave = threadIdx.x / kWave, threads = blockDim.x;
    int *offsets = lds + waves * a.experts, *totals = offsets + a.experts + 1, *firsts = totals + a.experts,
        *sums = firsts + a.experts, *tmp = sums + threads;
    for (int i = threadIdx.x; i < waves * a.experts; i += threads) lds[i] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * a.chunk;
    const uint32_t end = begin + a.chunk < a.slots ? begin + a.chunk : a.slots;
    uint32_t b, e;
    wave_share(begin, end, wave, waves, &b, &e);
    int slots[N];
    count_share(a, b, e, lds + wave * a.experts, slots);

    // a thread takes one expert and a run [b0, b1) of workgroups, `parts` runs
    // to an expert; more experts than threads take turns
    int wide = 16;
    while (wide < a.experts && wide < threads) wide *= 2;
    const int part = threadIdx.x / wide, parts = threads / wide, per = (a.blocks + parts - 1) / parts;
    const int b0 = part * per < a.blocks ? part * per : a.blocks, b1 = b0 + per < a.blocks ? b0 + per : a.blocks;
    for (int e0 = 0, base = 0; e0 < a.experts; e0 += wide) {
        const int x = e0 + threadIdx.x % wide;
        int sum = 0, mine = 0;       // mine: of the workgroups before this one
        if (x < a.experts) {
#pragma unroll 8
            for (int i = b0; i < b1; ++i) {
                const int n = a.counts[i * a.experts + x];
                sum += n;
                mine += i < static_cast<int>(blockIdx.x) ? n : 0;
            }
        }
        sums[threadIdx.x] = sum;
        __syncthreads();
        const bool first = part == 0 && x < a.experts;
        int total = 0, all = 0;
        if (first)
            for (int p = 0; p < parts; ++p) total += sums[p * wide + x - e0];
        const int size = padded(total, a.pad);
        const int to = base + scan_threads(first ? size : 0, tmp, &all);
        base += all;
        __syncthreads();             // sums have been read
        sums[threadIdx.x] = mine;
        __syncthreads();
        if (first) {
            int at = to - size;
            offsets[x] = at;
            offsets[x + 1] = to;     // the same value as its neighbour's own
            totals[x] = total;
            for (int p = 0; p < parts; ++p) at += sums[p * wide + x - e0];
            firsts[x] = at;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= a.experts; i += threads) a.offsets[i] = offsets[i];
    for (int x = threadIdx.x; x < a.experts; x += threads) counts_to_places(lds, a.experts, x, waves, firsts[x]);
    __syncthreads();
    place_share(a, b, e, lds + wave * a.experts, slots);
    fill_padding(a, offsets, totals);
}

// --------------------------------------------------------------------- rows

// Picks of a token whose rows are in flight together.
constexpr int kPicks = 8;

// Rows of a sorted buffer that stand for no slot, set to zero: L lanes look at
// `each` sorted rows at a time, up to kPadRows.  (With a whole workgroup to 8 rows
// of whatever length and number, 9627 tokens x 64 to 7 rows each took 11.0 us, not
// 4.4, and 64 x 5120 bytes to 6 rows 3.7, not 2.8.)
constexpr int kPadRows = 8;

struct Padding {
    const int32_t *order, *offsets;
    uint32_t rows;
    int experts, each;
};

template <int L, bool NT>
__device__ __forceinline__ void zero_row(char *row, size_t bytes) {
    const size_t whole = bytes / 16;
    for (size_t i = threadIdx.x % L; i < whole; i += L) store_vec<NT>(u32x4{0, 0, 0, 0}, row + 16 * i);
    for (size_t i = 16 * whole + threadIdx.x % L; i < bytes; i += L) row[i] = 0;
}

template <int L, class F>
__device__ __forceinline__ void for_padding(const Padding &q, uint32_t group, uint32_t groups, F f) {
    constexpr uint32_t kStep = kExpertThreads / L;
    const uint32_t used = static_cast<uint32_t>(q.offsets[q.experts]), share = q.each * kStep;
    const uint32_t end = used < q.rows ? used : q.rows;
    for (uint32_t p0 = group * share; p0 < end; p0 += groups * share) {
        const uint32_t p = p0 + threadIdx.x / L;
        bool padding[kPadRows];
#pragma unroll
        for (int i = 0; i < kPadRows; ++i) padding[i] = i < q.each && p + i * kStep < end && q.order[p + i * kStep] < 0;
#pragma unroll
        for (int i = 0; i < kPadRows; ++i)
            if (padding[i]) f(p + i * kStep);
    }
}

struct GatherArgs {
    const char *in, *scales;
    char *out, *scales_out;
    const int32_t *pos;
    size_t row_bytes, in_stride, out_stride;                 // bytes
    size_t scale_bytes, scales_stride, scales_out_stride;
    Padding pad;
    uint32_t tokens, rows;
    uint32_t pad_groups;     // leading workgroups, for the padding
    uint32_t splits;         // workgroups that share a token's row
    uint32_t units, scale_units;
    int k;
};

// A 16-byte unit of a row.  The last unit of a row that is not a whole number
// of them starts 16 bytes before the row's end: the bytes that it shares with
// its neighbour are written twice, with the same value.
__device__ __forceinline__ size_t unit_at(uint32_t i, size_t bytes) {
    const size_t o = 16 * static_cast<size_t>(i);
    return o + 16 <= bytes ? o : bytes - 16;
}

// L lanes per token (L = kExpertThreads: its units are also split over
// workgroups), one unit per lane.  The token's row is read once and stored k
// times, so the traffic is nearly all writes: 8191 tokens x 4096 to 8 rows each
// 98 us, 6.1 TB/s; 8192 x 4096 with one pick in eight here 19 us, 7.0 TB/s (26 with
// the places read through the scalar cache and looked at one by one).  Its own
// row is read through the caches: non-temporal loads of it took 116 us, not 99.
template <int L, bool NT>
__global__ __launch_bounds__(kExpertThreads) void gather_rows(GatherArgs a) {
    if (blockIdx.x < a.pad_groups) {
        for_padding<L>(a.pad, blockIdx.x, a.pad_groups, [&](uint32_t p) {
            zero_row<L, NT>(a.out + p * a.out_stride, a.row_bytes);
            if (a.scales_out != nullptr) zero_row<L, NT>(a.scales_out + p * a.scales_out_stride, a.scale_bytes);
        });
        return;
    }
    const uint32_t group = blockIdx.x - a.pad_groups;
    constexpr uint32_t kTokens = kExpertThreads / L;
    const uint32_t t = L == kExpertThreads ? group / a.splits : group * kTokens + threadIdx.x / L;
    const uint32_t split = L == kExpertThreads ? group % a.splits : 0;
    if (t >= a.tokens) return;
    const int32_t *pos = a.pos + static_cast<size_t>(t) * a.k;
    const uint32_t units = a.units + a.scale_units;
    const uint32_t i = split * kExpertThreads + threadIdx.x % L;
    const bool data = i < a.units, mine = i < units;
    const size_t bytes = data ? a.row_bytes : a.scale_bytes;
    const char *src = data ? a.in + t * a.in_stride : a.scales + t * a.scales_stride;
    char *dst = data ? a.out : a.scales_out;
    const size_t stride = data ? a.out_stride : a.scales_out_stride;
    const uint32_t u = data ? i : i - a.units;
    const size_t o = bytes >= 16 ? unit_at(u, bytes) : 0;
    u32x4 v = {0, 0, 0, 0};
    if (mine && bytes >= 16) v = load_vec<false>(src + o);
    const auto put = [&](uint32_t p) {
        if (bytes >= 16) {
            store_vec<NT>(v, dst + p * stride + o);
        } else {
            for (size_t b = 0; b < bytes; ++b) dst[p * stride + b] = src[b];
        }
    };
    if constexpr (L >= kWave) {
        // a lane holds a pick's place: they are read with the row, and picks
        // that go nowhere take no turn
        const int lane = threadIdx.x % kWave;
        const uint32_t p = lane < a.k ? static_cast<uint32_t>(pos[lane]) : ~0u;
        for (uint64_t left = __builtin_amdgcn_ballot_w64(p < a.rows); left != 0; left &= left - 1) {
            const uint32_t to = __builtin_amdgcn_readlane(p, __builtin_ctzll(left));
            if (mine) put(to);
        }
    } else {
        // the places first: they lie in memory that the stores could be thought
        // to change, and would be waited for one by one
        for (int j0 = 0; j0 < a.k; j0 += kPicks) {
            uint32_t p[kPicks];
#pragma unroll
            for (int j = 0; j < kPicks; ++j) p[j] = j0 + j < a.k ? static_cast<uint32_t>(pos[j0 + j]) : ~0u;
#pragma unroll
            for (int j = 0; j < kPicks; ++j)
                if (mine && p[j] < a.rows) put(p[j]);
        }
    }
}

struct CombineArgs {
    const uint16_t *z, *addend;
    uint16_t *out;
    const int32_t *pos;
    const float *weights;
    size_t z_stride, addend_stride, out_stride;              // values
    uint32_t tokens, rows;
    uint32_t splits;
    int k, hidden;
};

// The sum is binary32 and runs in pick order, the addend first; one rounding.
// L lanes per token (L = kExpertThreads: its units are also split over
// workgroups), U units of a lane at once.  Bound by HBM: 8191 tokens x 4096 of 8
// picks 101 us, 6.0 TB/s; 8192 x 4096 of 8 picks, one in eight of them here, 25
// (40 with the places read through the scalar cache and looked at one by one).
// Rows that pass the caches by are read by up to 6 waves of a SIMD, between what
// is best for rows that are all here (16384 x 4096 of 8 picks with 8, 6 and 4
// waves 207, 205 and 200 us) and for few of them (the 25 us above: 23, 25, 30).
template <class E, int L, int U, bool TAIL, bool NT>
__global__ __launch_bounds__(kExpertThreads)
__attribute__((amdgpu_waves_per_eu(1, NT && L >= kWave ? 6 : 8))) void combine_rows(CombineArgs a) {
    constexpr uint32_t kTokens = kExpertThreads / L;
    const uint32_t t = L == kExpertThreads ? blockIdx.x / a.splits : blockIdx.x * kTokens + threadIdx.x / L;
    const uint32_t split = L == kExpertThreads ? blockIdx.x % a.splits : 0;
    if (t >= a.tokens) return;
    const int32_t *pos = a.pos + static_cast<size_t>(t) * a.k;
    const float *weights = a.weights != nullptr ? a.weights + static_cast<size_t>(t) * a.k : nullptr;
    const int units = (a.hidden + 7) / 8;
    if constexpr (L >= kWave) {
        // A lane holds a pick's place and weight, so that both are read at
        // once and picks that go nowhere take no turn.  All lanes of a wave stay
        // to be asked for them: one without a unit loads the row's last.
        constexpr int kAtOnce = kPicks / U;
        const int lane = threadIdx.x % kWave;
        const uint32_t p = lane < a.k ? static_cast<uint32_t>(pos[lane]) : ~0u;
        const float w = weights != nullptr && lane < a.k ? weights[lane] : 1.0f;
        const int i0 = static_cast<int>(split) * kExpertThreads * U + threadIdx.x % L;
        if (i0 - lane >= units) return;
        const auto unit = [&](int u) {
            const int i = i0 + u * L;
            return Unit<TAIL>(i < units ? i : units - 1, a.hidden);
        };
        float sum[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            u32x4 x = {0, 0, 0, 0};
            if (a.addend != nullptr) x = unit(u).load(a.addend + t * a.addend_stride);
            Wide<E>::widen(x, sum[u]);
        }
        uint64_t left = __builtin_amdgcn_ballot_w64(p < a.rows);
        // (a full batch apart, whose rows are then added one by one as they come)
        const auto batch = [&](auto full) {
            u32x4 z[kAtOnce][U];
            float weight[kAtOnce];
            uint64_t next = left;
#pragma unroll
            for (int b = 0; b < kAtOnce; ++b) {
                if (!full && next == 0) break;
                const int from = __builtin_ctzll(next);
                next &= next - 1;
                const uint16_t *row = a.z + static_cast<uint32_t>(__builtin_amdgcn_readlane(p, from)) * a.z_stride;
                weight[b] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), from));
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u == 0 || i0 + u * L < units) z[b][u] = unit(u).template load<NT>(row);
            }
#pragma unroll
            for (int b = 0; b < kAtOnce; ++b) {
                if (!full && left == 0) break;
                left &= left - 1;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[8];
                    Wide<E>::widen(z[b][u], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[u][e] = fmaf(weight[b], f[e], sum[u][e]);
                }
            }
        };
        while (__builtin_popcountll(left) >= kAtOnce) batch(std::true_type{});
        while (left != 0) batch(std::false_type{});
#pragma unroll
        for (int u = 0; u < U; ++u)
            // its own values only: out may be the addend, which a neighbour reads
            if (i0 + u * L < units) unit(u).template store_own<NT>(a.out + t * a.out_stride, Wide<E>::narrow(sum[u]));
        return;
    }
    for (int i = threadIdx.x % L; i < units; i += L) {
        const Unit<TAIL> at(i, a.hidden);
        float sum[8];
        if (a.addend != nullptr) {
            Wide<E>::widen(at.load(a.addend + t * a.addend_stride), sum);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
        }
        for (int j0 = 0; j0 < a.k; j0 += kPicks) {
            u32x4 z[kPicks];
            float w[kPicks];
            bool there[kPicks];
#pragma unroll
            for (int j = 0; j < kPicks; ++j) {
                there[j] = false;
                if (j0 + j < a.k) {
                    const uint32_t p = static_cast<uint32_t>(pos[j0 + j]);
                    there[j] = p < a.rows;
                    if (there[j]) {
                        z[j] = at.template load<NT>(a.z + p * a.z_stride);
                        w[j] = weights != nullptr ? weights[j0 + j] : 1.0f;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kPicks; ++j) {
                if (there[j]) {
                    float f[8];
                    Wide<E>::widen(z[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[j], f[e], sum[e]);
                }
            }
        }
        at.template store_own<NT>(a.out + t * a.out_stride, Wide<E>::narrow(sum));
    }
}

struct CombineGradArgs {
    const uint16_t *dy, *z;
    uint16_t *dz;
    const int32_t *pos;
    const float *weights;
    float *dweights;
    size_t dy_stride, z_stride, dz_stride;                   // values
    Padding pad;
    uint32_t tokens, rows;
    uint32_t pad_groups;
    int k, hidden;
};

// L lanes per token over all of its row, since the weights' gradients are sums
// over it; kPicks of them at a time in registers.  Bound by HBM: 4096 tokens x
// 8192 of 4 picks 118 us, 630 MB with the padding, 5.3 TB/s; 8192 x 4096 with one
// pick in eight here 32 us (44 with the places read through the scalar cache).
template <class E, int L, bool TAIL, bool NT>
__global__ __launch_bounds__(kExpertThreads) void combine_grad_rows(CombineGradArgs a) {
    __shared__ float sums[kExpertThreads / kWave][kPicks];
    if (blockIdx.x < a.pad_groups) {
        for_padding<L>(a.pad, blockIdx.x, a.pad_groups, [&](uint32_t p) {
            zero_row<L, NT>(reinterpret_cast<char *>(a.dz + p * a.dz_stride), static_cast<size_t>(a.hidden) * 2);
        });
        return;
    }
    constexpr uint32_t kTokens = kExpertThreads / L;
    const uint32_t group = blockIdx.x - a.pad_groups;
    const uint32_t t = group * kTokens + (L == kExpertThreads ? 0 : threadIdx.x / L);
    const int lane = static_cast<int>(threadIdx.x) % L;
    const bool here = t < a.tokens;
    const int32_t *pos = a.pos + static_cast<size_t>(t) * a.k;
    const int units = here ? (a.hidden + 7) / 8 : 0;
    // (a lane holds a pick's place and weight, which are read at once)
    const int pick = threadIdx.x % kWave;
    uint32_t place = ~0u;
    float weight = 1.0f;
    if (L >= kWave && here && pick < a.k) {
        place = static_cast<uint32_t>(pos[pick]);
        if (a.weights != nullptr) weight = a.weights[static_cast<size_t>(t) * a.k + pick];
    }
    for (int j0 = 0; j0 < a.k; j0 += kPicks) {
        uint32_t p[kPicks];
        float w[kPicks], dot[kPicks];
#pragma unroll
        for (int j = 0; j < kPicks; ++j) {
            p[j] = ~0u;
            w[j] = 1.0f;
            dot[j] = 0.0f;
            if constexpr (L >= kWave) {
                p[j] = static_cast<uint32_t>(__builtin_amdgcn_readlane(place, j0 + j));
                w[j] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), j0 + j));
            } else if (here && j0 + j < a.k) {
                p[j] = static_cast<uint32_t>(pos[j0 + j]);
                if (a.weights != nullptr) w[j] = a.weights[static_cast<size_t>(t) * a.k + j0 + j];
            }
        }
        for (int i = lane; i < units; i += L) {
            const Unit<TAIL> at(i, a.hidden);
            float d[8];
            u32x4 z[kPicks];
            Wide<E>::widen(at.load(a.dy + t * a.dy_stride), d);
            if (a.dweights != nullptr) {
#pragma unroll
                for (int j = 0; j < kPicks; ++j)
                    if (p[j] < a.rows) z[j] = at.template load<NT>(a.z + p[j] * a.z_stride);
            }
#pragma unroll
            for (int j = 0; j < kPicks; ++j) {
                if (p[j] < a.rows) {
                    float f[8];
                    if (a.dweights != nullptr) {
                        Wide<E>::widen(z[j], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dot[j] = at.own(e) ? fmaf(d[e], f[e], dot[j]) : dot[j];
                    }
                    if (a.dz != nullptr) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = d[e] * w[j];
                        // its own values only: dz may be z, which a neighbour reads
                        at.template store_own<NT>(a.dz + p[j] * a.dz_stride, Wide<E>::narrow(f));
                    }
                }
            }
        }
        if (a.dweights == nullptr) continue;
        if constexpr (L <= kWave) {
#pragma unroll
            for (int j = 0; j < kPicks; ++j) {
                dot[j] = sum_lanes<L>(dot[j]);
                if (here && lane == j && j0 + j < a.k) a.dweights[static_cast<size_t>(t) * a.k + j0 + j] = dot[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPicks; ++j) {
                dot[j] = sum_lanes<kWave>(dot[j]);
                if (threadIdx.x % kWave == 0) sums[threadIdx.x / kWave][j] = dot[j];
            }
            __syncthreads();
            if (here && threadIdx.x < kPicks && j0 + static_cast<int>(threadIdx.x) < a.k) {
                float s = sums[0][threadIdx.x];
#pragma unroll
                for (int v = 1; v < kExpertThreads / kWave; ++v) s += sums[v][threadIdx.x];
                a.dweights[static_cast<size_t>(t) * a.k + j0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

namespace {

constexpr size_t kMaxCount = 0x7FFFFFFF;
// A launch has fewer than 2^32 work-items.
constexpr size_t kMaxGroups = 0xFFFFFFFFu / kExpertThreads;
constexpr size_t kSortBlocks = 256;
constexpr size_t kSortChunk = 2048;
constexpr int kSortBatch = 8;

// Workgroups for the padding.  Few rows are spread over them before a lane takes
// a second one (gathers with 512, 1024 and 2048: 955 tokens x 512 bytes to 4 rows
// padded to 64 3.6, 3.1 and 3.5 us; 64 x 4096 to 8 rows of 512 experts 5.7, 5.8
// and 6.3), and many take turns in them (8191 tokens x 4096 to 8 rows, none of them
// padding, with 1024, 2048 and 2^18: 104.5, 110.8 and 112.9 us, 105.4 unasked;
// 2000 x 4096 to 8 rows padded to 64, 32 us in all three).
constexpr size_t kPadGroups = 1024;

uint32_t sort_chunk(size_t slots) {
    const size_t c = (slots + kSortBlocks - 1) / kSortBlocks;
    return static_cast<uint32_t>(c < kSortChunk ? kSortChunk : (c + kWave - 1) / kWave * kWave);
}

bool picks_ok(size_t tokens, int k, size_t *slots) {
    return k >= 1 && !__builtin_mul_overflow(tokens, static_cast<size_t>(k), slots);
}

// Rows that a sort of so many slots takes at most: pad - 1 beside them for every
// segment that can hold one.  False above what hr_experts_sort takes.
bool sort_rows(size_t slots, int k, int experts, int pad, size_t *rows) {
    if (k > HR_EXPERTS_MAX_K || experts > HR_EXPERTS_MAX || slots > kMaxCount) return false;
    const size_t segments = static_cast<size_t>(experts) < slots ? static_cast<size_t>(experts) : slots;
    *rows = slots + segments * static_cast<size_t>(pad - 1);     // below 2^42
    return *rows <= kMaxCount;
}

// Lanes that a row of `units` 16-byte units keeps busy.
int lanes_for(size_t units) { return units <= 16 ? 16 : units <= 64 ? 64 : kExpertThreads; }

// Sorted rows of this many bytes or more pass the caches by (non-temporal
// loads and stores).  Measured cached and streamed, as a sort, a gather and a
// combine of 8 picks of 4096 values on three sets of buffers in turn: 33 MB of
// rows 23.7 and 24.2 us, 67 MB 51.3 and 41.7, 134 MB 77.2 and 62.9, 537 MB 277
// and 209.  On one set, a copy in the place of the experts' products between
// gather and combine: 33 MB 37 and 42 in all, 67 MB 58 and 64, 134 MB 135 and
// 121, 537 MB 527 and 473.
constexpr size_t kStreamBytes = size_t(1) << 26;

template <class K, class A>
hipError_t launch_k(K k, size_t grid, hipStream_t s, const A &a) {
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(grid)), dim3(kExpertThreads), 0, s, a);
    return hipGetLastError();
}

// Workgroups of the padding beside `others`, for every row that an order comes
// with.  (The buffer's size says nothing: the segments of a rank's share of the
// picks are padded and still fit into fewer rows than there are slots.)
uint32_t padding_groups(Padding &q, int lanes, size_t others) {
    if (q.order == nullptr) return 0;
    const size_t at_once = kExpertThreads / lanes, each = q.rows / (at_once * kPadGroups) + 1;
    q.each = each < kPadRows ? static_cast<int>(each) : kPadRows;
    const size_t rows = at_once * q.each, groups = (q.rows + rows - 1) / rows;
    const size_t room = others + kPadGroups < kMaxGroups ? kPadGroups : kMaxGroups - others;
    return static_cast<uint32_t>(groups < room ? groups : room);
}

// The variant of a kernel for a call's `tail` and `nt`.
#define HR_VARIANT(K, ...)                                                                  \
    (tail ? (nt ? K<E, __VA_ARGS__, true, true> : K<E, __VA_ARGS__, true, false>)           \
          : (nt ? K<E, __VA_ARGS__, false, true> : K<E, __VA_ARGS__, false, false>))

template <class E>
hr_status combine_impl(const hr_experts_combine_args *q, hr_stream_t stream) {
    size_t slots = 0;
    if (q == nullptr || q->hidden == 0 || q->k > HR_EXPERTS_MAX_K || !picks_ok(q->tokens, q->k, &slots))
        return HR_ERR_INVALID_ARG;
    if (slots > kMaxCount || q->rows > kMaxCount || q->hidden > kMaxCount / 16) return HR_ERR_TOO_LARGE;
    if (q->tokens == 0) return HR_OK;
    if (q->pos == nullptr || q->out == nullptr || (q->z == nullptr && q->rows > 0)) return HR_ERR_INVALID_ARG;
    CombineArgs a{};
    a.z_stride = q->z_stride;
    a.addend_stride = q->addend_stride;
    a.out_stride = q->out_stride;
    if (!row_stride(q->rows, q->hidden, &a.z_stride, 2) || !row_stride(q->tokens, q->hidden, &a.addend_stride, 2) ||
        !row_stride(q->tokens, q->hidden, &a.out_stride, 2))
        return HR_ERR_INVALID_ARG;
    if (!aligned(q->z, 2) || !aligned(q->addend, 2) || !aligned(q->out, 2) || !aligned(q->pos, 4) ||
        !aligned(q->weights, 4))
        return HR_ERR_ALIGNMENT;
    const size_t width = q->hidden * 2, per = static_cast<size_t>(q->k) * 4;
    const Region out = {q->out, q->tokens, width, a.out_stride * 2};
    const Region addend = {q->addend, q->tokens, width, a.addend_stride * 2};
    if (regions_overlap(out, {q->z, q->rows, width, a.z_stride * 2}) ||
        regions_overlap(out, {q->pos, q->tokens, per, per}) || regions_overlap(out, {q->weights, q->tokens, per, per}) ||
        (regions_overlap(out, addend) && !regions_same(out, addend)))
        return HR_ERR_INVALID_ARG;
    a.z = static_cast<const uint16_t *>(q->z);
    a.addend = static_cast<const uint16_t *>(q->addend);
    a.out = static_cast<uint16_t *>(q->out);
    a.pos = q->pos;
    a.weights = q->weights;
    a.tokens = static_cast<uint32_t>(q->tokens);
    a.rows = static_cast<uint32_t>(q->rows);
    a.k = q->k;
    a.hidden = static_cast<int>(q->hidden);
    const size_t units = (q->hidden + 7) / 8;
    const int lanes = lanes_for(units);
    // two units of a lane where a second workgroup would have less than half of
    // its lanes busy (8192 tokens x 2304 of 2 picks 28.6 and 23.2 us; with two
    // full workgroups of such a token's row the second unit only costs waves)
    const int at_once = units > kExpertThreads && units < kExpertThreads * 3 / 2 ? 2 : 1;
    const size_t share = static_cast<size_t>(kExpertThreads) * at_once;
    a.splits = lanes == kExpertThreads ? static_cast<uint32_t>((units + share - 1) / share) : 1;
    const size_t grid = lanes == kExpertThreads ? q->tokens * a.splits
                                                : (q->tokens + kExpertThreads / lanes - 1) / (kExpertThreads / lanes);
    if (grid > kMaxGroups) return HR_ERR_TOO_LARGE;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool nt = slots * width >= kStreamBytes, tail = q->hidden % 8 != 0;
    const hipError_t e = lanes == 16    ? launch_k(HR_VARIANT(combine_rows, 16, 1), grid, s, a)
                         : lanes == 64  ? launch_k(HR_VARIANT(combine_rows, 64, 1), grid, s, a)
                         : at_once == 1 ? launch_k(HR_VARIANT(combine_rows, kExpertThreads, 1), grid, s, a)
                                        : launch_k(HR_VARIANT(combine_rows, kExpertThreads, 2), grid, s, a);
    return e == hipSuccess ? HR_OK : HR_ERR_HIP;
}

template <class E>
hr_status combine_grad_impl(const hr_experts_combine_grad_args *q, hr_stream_t stream) {
    size_t slots = 0;
    if (q == nullptr || q->hidden == 0 || q->k > HR_EXPERTS_MAX_K || !picks_ok(q->tokens, q->k, &slots))
        return HR_ERR_INVALID_ARG;
    if (q->dz == nullptr && q->dweights == nullptr) return q->tokens == 0 ? HR_OK : HR_ERR_INVALID_ARG;
    if (slots > kMaxCount || q->rows > kMaxCount || q->hidden > kMaxCount / 16) return HR_ERR_TOO_LARGE;
    if (q->order != nullptr && (q->offsets == nullptr || q->experts < 1)) return HR_ERR_INVALID_ARG;
    if (q->tokens == 0) return HR_OK;
    if (q->pos == nullptr || q->dy == nullptr) return HR_ERR_INVALID_ARG;
    if (q->dweights != nullptr && q->z == nullptr && q->rows > 0) return HR_ERR_INVALID_ARG;
    CombineGradArgs a{};
    a.dy_stride = q->dy_stride;
    a.z_stride = q->z_stride;
    a.dz_stride = q->dz_stride;
    if (!row_stride(q->tokens, q->hidden, &a.dy_stride, 2) || !row_stride(q->rows, q->hidden, &a.z_stride, 2) ||
        !row_stride(q->rows, q->hidden, &a.dz_stride, 2))
        return HR_ERR_INVALID_ARG;
    if (!aligned(q->dy, 2) || !aligned(q->z, 2) || !aligned(q->dz, 2) || !aligned(q->pos, 4) ||
        !aligned(q->weights, 4) || !aligned(q->dweights, 4) || !aligned(q->order, 4) || !aligned(q->offsets, 4))
        return HR_ERR_ALIGNMENT;
    const size_t width = q->hidden * 2, per = static_cast<size_t>(q->k) * 4;
    const Region dz = {q->dz, q->rows, width, a.dz_stride * 2}, dw = {q->dweights, q->tokens, per, per};
    const Region z = {q->dweights != nullptr ? q->z : nullptr, q->rows, width, a.z_stride * 2};
    const Region ins[] = {{q->dy, q->tokens, width, a.dy_stride * 2},
                          {q->pos, q->tokens, per, per},
                          {q->weights, q->tokens, per, per},
                          {q->order, 1, q->rows * 4, 0},
                          {q->offsets, 1, (static_cast<size_t>(q->experts > 0 ? q->experts : 0) + 1) * 4, 0}};
    for (const Region &r : ins)
        if (regions_overlap(dz, r) || regions_overlap(dw, r)) return HR_ERR_INVALID_ARG;
    if (regions_overlap(dz, dw) || regions_overlap(dw, z) || (regions_overlap(dz, z) && !regions_same(dz, z)))
        return HR_ERR_INVALID_ARG;
    a.dy = static_cast<const uint16_t *>(q->dy);
    a.z = static_cast<const uint16_t *>(q->z);
    a.dz = static_cast<uint16_t *>(q->dz);
    a.pos = q->pos;
    a.weights = q->weights;
    a.dweights = q->dweights;
    a.pad = Padding{q->dz != nullptr ? q->order : nullptr, q->offsets, static_cast<uint32_t>(q->rows), q->experts, 1};
    a.tokens = static_cast<uint32_t>(q->tokens);
    a.rows = static_cast<uint32_t>(q->rows);
    a.k = q->k;
    a.hidden = static_cast<int>(q->hidden);
    const int lanes = lanes_for((q->hidden + 7) / 8);
    const size_t groups = (q->tokens + kExpertThreads / lanes - 1) / (kExpertThreads / lanes);
    if (groups + (a.pad.order != nullptr) > kMaxGroups) return HR_ERR_TOO_LARGE;
    a.pad_groups = padding_groups(a.pad, lanes, groups);
    const size_t grid = a.pad_groups + groups;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool nt = slots * width >= kStreamBytes, tail = q->hidden % 8 != 0;
    const hipError_t e = lanes == 16   ? launch_k(HR_VARIANT(combine_grad_rows, 16), grid, s, a)
                         : lanes == 64 ? launch_k(HR_VARIANT(combine_grad_rows, 64), grid, s, a)
                                       : launch_k(HR_VARIANT(combine_grad_rows, kExpertThreads), grid, s, a);
    return e == hipSuccess ? HR_OK : HR_ERR_HIP;
}

#undef HR_VARIANT

}  // namespace

}  // namespace hr

using namespace hr;

extern "C" HR_API size_t hr_experts_rows(size_t tokens, int k, int experts, int pad) {
    size_t slots = 0, rows = 0;
    if (!picks_ok(tokens, k, &slots) || experts < 1 || pad < 1) return 0;
    return sort_rows(slots, k, experts, pad, &rows) ? rows : 0;
}

extern "C" HR_API size_t hr_experts_sort_workspace(size_t tokens, int k, int experts) {
    size_t slots = 0;
    if (!picks_ok(tokens, k, &slots) || k > HR_EXPERTS_MAX_K || experts < 1 || experts > HR_EXPERTS_MAX ||
        slots > kMaxCount)
        return 0;
    if (slots <= static_cast<size_t>(HR_EXPERTS_SORT_FEW)) return 0;
    const size_t chunk = sort_chunk(slots);
    return (slots + chunk - 1) / chunk * static_cast<size_t>(experts) * 4;
}

extern "C" HR_API hr_status hr_experts_sort(const int32_t *ids, size_t tokens, int k, int first, int experts, int pad,
                                            int32_t *offsets, int32_t *order, size_t rows, int32_t *pos,
                                            void *workspace, size_t workspace_bytes, hr_stream_t stream) {
    size_t slots = 0;
    if (!picks_ok(tokens, k, &slots) || first < 0 || experts < 1 || pad < 1) return HR_ERR_INVALID_ARG;
    size_t most = 0;
    if (!sort_rows(slots, k, experts, pad, &most) || rows > kMaxCount) return HR_ERR_TOO_LARGE;
    if (rows < most) return HR_ERR_INVALID_ARG;
    if (offsets == nullptr || (rows > 0 && order == nullptr) || (slots > 0 && (ids == nullptr || pos == nullptr)))
        return HR_ERR_INVALID_ARG;
    const size_t need = hr_experts_sort_workspace(tokens, k, experts);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return HR_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(pos, 4) || !aligned(workspace, 4))
        return HR_ERR_ALIGNMENT;
    const Region all[] = {{ids, 1, slots * 4, 0},
                          {offsets, 1, (static_cast<size_t>(experts) + 1) * 4, 0},
                          {order, 1, rows * 4, 0},
                          {pos, 1, slots * 4, 0},
                          {workspace, 1, need, 0}};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (regions_overlap(all[i], all[j])) return HR_ERR_INVALID_ARG;

    SortArgs a{};
    a.ids = ids;
    a.offsets = offsets;
    a.order = order;
    a.pos = pos;
    a.counts = static_cast<int32_t *>(workspace);
    a.slots = static_cast<uint32_t>(slots);
    a.rows = static_cast<uint32_t>(rows);
    a.first = first;
    a.experts = experts;
    a.pad = pad;
    while ((1 << a.bits) <= experts) ++a.bits;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    // 16 waves' counts of up to 512 experts, or 8 waves' of up to 1024
    const int most_threads = experts <= 512 ? 1024 : 512;
    const auto lds_for = [&](int threads, int arrays, int more) {
        return (static_cast<size_t>(threads / kWave + arrays) * experts + 1 + more + threads / kWave) * sizeof(int);
    };
    // The kernel for 1 or 2 slots of a thread where that many do: the code of
    // eight costs small calls 0.3 us.
    const auto launch = [&](auto one, auto two, auto many, size_t chunk, int blocks, int threads, size_t lds) {
        const size_t each = (chunk + threads - 1) / threads;
        hipLaunchKernelGGL(each <= 1 ? one : each <= 2 ? two : many, dim3(blocks), dim3(threads), lds, s, a);
    };
    if (slots <= static_cast<size_t>(HR_EXPERTS_SORT_FEW)) {
        // a wave for every 64 slots, but no fewer than 4
        int threads = 256;
        while (threads < most_threads && threads < static_cast<int>(slots)) threads *= 2;
        launch(sort_once<1>, sort_once<2>, sort_once<kSortBatch>, slots, 1, threads, lds_for(threads, 2, 0));
        return hipGetLastError() == hipSuccess ? HR_OK : HR_ERR_HIP;
    }
    a.chunk = sort_chunk(slots);
    a.blocks = static_cast<int>((slots + a.chunk - 1) / a.chunk);
    launch(sort_count<2>, sort_count<2>, sort_count<kSortBatch>, a.chunk, a.blocks, kMaxSortThreads,
           static_cast<size_t>(experts) * 4);
    if (hipGetLastError() != hipSuccess) return HR_ERR_HIP;
    launch(sort_place<2>, sort_place<2>, sort_place<kSortBatch>, a.chunk, a.blocks, most_threads,
           lds_for(most_threads, 3, most_threads));
    return hipGetLastError() == hipSuccess ? HR_OK : HR_ERR_HIP;
}

extern "C" HR_API hr_status hr_experts_gather(const hr_experts_gather_args *q, hr_stream_t stream) {
    size_t slots = 0;
    if (q == nullptr || q->row_bytes == 0 || q->k > HR_EXPERTS_MAX_K || !picks_ok(q->tokens, q->k, &slots))
        return HR_ERR_INVALID_ARG;
    if (slots > kMaxCount || q->rows > kMaxCount || q->row_bytes > kMaxCount || q->scales_width > kMaxCount / 4)
        return HR_ERR_TOO_LARGE;
    if ((q->scales == nullptr) != (q->scales_out == nullptr) && q->tokens > 0 && q->rows > 0) return HR_ERR_INVALID_ARG;
    if (q->scales != nullptr && q->scales_width == 0) return HR_ERR_INVALID_ARG;
    if (q->order != nullptr && (q->offsets == nullptr || q->experts < 1)) return HR_ERR_INVALID_ARG;
    if (q->tokens == 0 || q->rows == 0) return HR_OK;
    if (q->in == nullptr || q->out == nullptr || q->pos == nullptr) return HR_ERR_INVALID_ARG;
    GatherArgs a{};
    a.in_stride = q->in_stride;
    a.out_stride = q->out_stride;
    size_t ss = q->scales_stride, so = q->scales_out_stride;
    if (!row_stride(q->tokens, q->row_bytes, &a.in_stride, 1) || !row_stride(q->rows, q->row_bytes, &a.out_stride, 1) ||
        !row_stride(q->tokens, q->scales_width, &ss, 4) || !row_stride(q->rows, q->scales_width, &so, 4))
        return HR_ERR_INVALID_ARG;
    if (!aligned(q->pos, 4) || !aligned(q->scales, 4) || !aligned(q->scales_out, 4) || !aligned(q->order, 4) ||
        !aligned(q->offsets, 4))
        return HR_ERR_ALIGNMENT;
    const size_t per = static_cast<size_t>(q->k) * 4;
    const Region out = {q->out, q->rows, q->row_bytes, a.out_stride};
    const Region sout = {q->scales_out, q->rows, q->scales_width * 4, so * 4};
    const Region ins[] = {{q->in, q->tokens, q->row_bytes, a.in_stride},
                          {q->scales, q->tokens, q->scales_width * 4, ss * 4},
                          {q->pos, q->tokens, per, per},
                          {q->order, 1, q->rows * 4, 0},
                          {q->offsets, 1, (static_cast<size_t>(q->experts > 0 ? q->experts : 0) + 1) * 4, 0}};
    for (const Region &r : ins)
        if (regions_overlap(out, r) || regions_overlap(sout, r)) return HR_ERR_INVALID_ARG;
    if (regions_overlap(out, sout)) return HR_ERR_INVALID_ARG;

    a.in = static_cast<const char *>(q->in);
    a.out = static_cast<char *>(q->out);
    a.pos = q->pos;
    a.row_bytes = q->row_bytes;
    a.units = static_cast<uint32_t>((q->row_bytes + 15) / 16);
    if (q->scales != nullptr) {
        a.scales = reinterpret_cast<const char *>(q->scales);
        a.scales_out = reinterpret_cast<char *>(q->scales_out);
        a.scale_bytes = q->scales_width * 4;
        a.scales_stride = ss * 4;
        a.scales_out_stride = so * 4;
        a.scale_units = static_cast<uint32_t>((a.scale_bytes + 15) / 16);
    }
    a.pad = Padding{q->order, q->offsets, static_cast<uint32_t>(q->rows), q->experts, 1};
    a.tokens = static_cast<uint32_t>(q->tokens);
    a.rows = static_cast<uint32_t>(q->rows);
    a.k = q->k;
    const size_t units = static_cast<size_t>(a.units) + a.scale_units;
    const int lanes = lanes_for(units);
    a.splits = lanes == kExpertThreads ? static_cast<uint32_t>((units + kExpertThreads - 1) / kExpertThreads) : 1;
    const size_t groups = lanes == kExpertThreads ? q->tokens * a.splits
                                                  : (q->tokens + kExpertThreads / lanes - 1) / (kExpertThreads / lanes);
    if (groups + (a.pad.order != nullptr) > kMaxGroups) return HR_ERR_TOO_LARGE;
    a.pad_groups = padding_groups(a.pad, lanes, groups);
    const size_t grid = a.pad_groups + groups;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool nt = slots * (q->row_bytes + a.scale_bytes) >= kStreamBytes;
    const hipError_t e = lanes == 16   ? launch_k(nt ? gather_rows<16, true> : gather_rows<16, false>, grid, s, a)
                         : lanes == 64 ? launch_k(nt ? gather_rows<64, true> : gather_rows<64, false>, grid, s, a)
                                       : launch_k(nt ? gather_rows<kExpertThreads, true>
                                                     : gather_rows<kExpertThreads, false>, grid, s, a);
    return e == hipSuccess ? HR_OK : HR_ERR_HIP;
}

extern "C" HR_API hr_status hr_experts_combine_f16(const hr_experts_combine_args *args, hr_stream_t stream) {
    return combine_impl<F16>(args, stream);
}

extern "C" HR_API hr_status hr_experts_combine_bf16(const hr_experts_combine_args *args, hr_stream_t stream) {
    return combine_impl<BF16>(args, stream);
}

extern "C" HR_API hr_status hr_experts_combine_grad_f16(const hr_experts_combine_grad_args *args, hr_stream_t stream) {
    return combine_grad_impl<F16>(args, stream);
}

extern "C" HR_API hr_status hr_experts_combine_grad_bf16(const hr_experts_combine_grad_args *args,
                                                         hr_stream_t stream) {
    return combine_grad_impl<BF16>(args, stream);
}
