// product.h -- the tile kernel behind the experts' products; not exported.
//
//   out[q][p] = sum over c of Q[q][c] * P[p][c]
//
// The rows of `out` run over q, its adjacent values over p:
//
//   product                       q: sorted rows   p: n   c: k   P = w, as it lies
//   product, transposed matrices  q: sorted rows   p: n   c: k   P = w, strided in c
//   weights' gradient             q: n             p: k   c: a segment's rows,
//                                                         both strided in c
//
// An operand is "along" when its adjacent values run over c, and "across" when
// they run over q or p.  A panel of an operand is B rows of 128 bytes of c
// (along) or 128 bytes' worth of c rows of B values (across); panels go from HBM
// to LDS by 16-byte DMA, with no register between, several stages ahead.
//
// LDS.  64 banks of 4 bytes: 16 lanes of a 16-byte read, or 32 lanes of an
// 8-byte one, should touch 256 different bytes of a 256-byte line.  Rows of
// an along panel are 128 bytes apart, so the 16 rows that a matrix
// instruction's operand wants lie 8 deep on the same banks; unit u of row r
// is therefore kept at place u ^ h(r), with h taking 8 values over 16 rows of
// either parity.  Across panels are read transposed (ds_read_b64_tr), 8 or 16
// rows at a time, and their slots are moved by the row in the same way.  DMA
// writes 64 consecutive units, so the lanes' global addresses carry the move.
//
// Matrix instructions.  16 x 16 x 32 (16 bits) and 16 x 16 x 128 (e4m3), P as
// the first operand: a lane then holds four adjacent values of one row of
// out.  The order of c inside an instruction is the same for both operands
// and otherwise free: lanes 16 g .. 16 g + 15 take units g and g + 4 of a panel.
// The rows of P that make up an operand are free too: those of four operands
// are interleaved by four, so that a lane's four times four values are adjacent.
//
// e4m3.  A panel is one group of 128, so one instruction's result, in binary32,
// is scaled by the row's scale times the block's and added to the sum in binary32.
// (The instruction itself adds the products of its groups of 8 after cutting
// them at 2^-13 of the largest's leading bit, measured; products of two e4m3
// values have 8 bits.  The 16-bit instructions keep all of binary32.)
#pragma once

#include <type_traits>

#include "rows.h"

namespace hr {

struct E4M3 {};

template <class E>
constexpr int kBytes = 2;
template <>
inline constexpr int kBytes<E4M3> = 1;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

#define HR_LDS __attribute__((address_space(3)))

struct ProductArgs {
    const char *q, *p;
    char *out;
    const int32_t *offsets;             // NULL: one segment of all rows
    const float *q_scales, *p_scales;   // e4m3
    size_t q_stride, p_stride, out_stride;          // bytes between rows as they lie
    size_t p_expert_stride, out_expert_stride;      // bytes
    size_t q_scales_stride;                         // scales between rows
    size_t scales_expert, scales_p, scales_c;       // scales between experts, blocks of p and of c
    uint32_t rows;
    int experts;
    int nq, np, nc;                     // extents of q (gradient), p and c (product)
    int tiles_q, tiles_p;               // tiles_q: of the gradient
    int stream;                         // out passes the caches by
};

// One stage's place in a lane's address: 16 bytes from `offset` past the
// base; a lane whose offset is kNowhere reads zeros and touches no memory
// (the buffer's bounds check).
constexpr uint32_t kNowhere = 0x80000000u;

__device__ __forceinline__ i32x4 buffer_of(const char *base, bool here = true) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    return i32x4{static_cast<int>(a), static_cast<int>((a >> 32) & 0xFFFFu), here ? 0x7FFFFFFF : 0, 0x00020000};
}

// 16 (or 4) bytes a lane from HBM to LDS at `to` + 16 (4) * lane.  Written out
// because the compiler, seeing the builtin, waits for every load in flight
// before any LDS read; nothing here lands in registers.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"     // (m0 is reserved: the compiler writes it again before its own uses)
__device__ __forceinline__ void dma16(i32x4 from, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(offset), "s"(from)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(i32x4 from, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(offset), "s"(from)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// All but the last N loads have landed, and this wave's LDS reads are done.
template <int N>
__device__ __forceinline__ void landed() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ void meet() { asm volatile("s_barrier" : : : "memory"); }

// The LDS reads above are done, and nothing moves over this line.
__device__ __forceinline__ void read_done() {
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void change() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// A value that no kernel running now writes, at an address that a wave shares:
// read through the scalar cache, so that it is not waited for with the loads.
__device__ __forceinline__ float constant_at(const float *p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) float *>(reinterpret_cast<uint64_t>(p));
}

template <class V>
__device__ __forceinline__ V lds_read(uint32_t at) {
    return *reinterpret_cast<const HR_LDS V *>(at);
}

// Where an operand's panel lies in LDS and in memory.  B: its rows or columns.
template <int SIZE, int B, bool ACROSS, bool INTERLEAVED>
struct Panel {
    static constexpr int kUnit = 16 / SIZE;             // values per unit
    static constexpr int kC = 128 / SIZE;               // values of c
    static constexpr int kPitch = ACROSS ? B * SIZE : 128;
    static constexpr int kBytesAll = B * 128;
    static constexpr int kDmas = kBytesAll / 1024;      // of a wave
    static constexpr int kRowsPerDma = 1024 / kPitch;

    // along: the move of row r's units
    static __device__ __forceinline__ uint32_t move_along(uint32_t r) {
        return INTERLEAVED ? ((r >> 1) & 1) | ((r >> 4) & 3) << 1 : (r >> 1) & 7;
    }
    // across: the move of row c's slots of 32 (16-bit) or 16 (e4m3) bytes
    static constexpr int kSlot = SIZE == 2 ? 32 : 16;
    static __device__ __forceinline__ uint32_t move_across(uint32_t c) {
        constexpr int shared = kPitch >= 256 ? 0 : kPitch == 128 ? 1 : kPitch == 64 ? 2 : kPitch == 32 ? 3 : 4;
        return (SIZE == 2 ? (c & 3) | ((c >> 3) & 1) << 2 : (c & 7) | ((c >> 4) & 1) << 3) >> shared;
    }

    // What lane l brings in DMA t of a panel: row `row` (of B, or of c) and unit
    // `unit` of it.
    static __device__ __forceinline__ void source(int t, uint32_t lane, uint32_t &row, uint32_t &unit) {
        const uint32_t byte = lane * 16;
        row = t * kRowsPerDma + byte / kPitch;
        const uint32_t at = byte % kPitch / 16;
        if constexpr (!ACROSS) {
            unit = at ^ move_along(row);
        } else if constexpr (SIZE == 2) {
            unit = ((at >> 1) ^ move_across(row)) << 1 | (at & 1);
        } else {
            unit = at ^ move_across(row);
        }
    }
    // Whether that unit is there, with b rows (columns) and c values of c left.
    static __device__ __forceinline__ bool there(uint32_t row, uint32_t unit, int b, int c) {
        const int r = static_cast<int>(row), u = static_cast<int>(unit) * kUnit;
        return ACROSS ? r < c && u < b : r < b && u < c;
    }
};

// A wave's reads of an operand from a panel in LDS: FRAGS operands of 16 rows
// from row `first` on, 32 bytes of c a lane (two 16-byte units).
template <int SIZE, int B, bool ACROSS, bool INTERLEAVED, int FRAGS>
struct Reader {
    using P = Panel<SIZE, B, ACROSS, INTERLEAVED>;
    uint32_t at[ACROSS ? FRAGS : 2];

    __device__ __forceinline__ void init(uint32_t first, uint32_t lane) {
        const uint32_t i = lane & 15, g = lane >> 4;
        if constexpr (!ACROSS) {
            const uint32_t r = INTERLEAVED ? first + 16 * (i >> 2) + (i & 3) : first + i;
            at[0] = r * 128 + ((g ^ P::move_along(r)) << 4);
            at[1] = at[0] ^ 64;
        } else {
            const uint32_t c = SIZE == 2 ? 8 * g + (i >> 2) : 16 * g + (i >> 1);
            const uint32_t sub = SIZE == 2 ? 8 * (i & 3) : 8 * (i & 1);
#pragma unroll
            for (int f = 0; f < FRAGS; ++f)
                at[f] = c * P::kPitch + (((first * SIZE / P::kSlot + f) ^ P::move_across(c)) * P::kSlot) + sub;
        }
    }
    // 16 bytes of c of operand f, unit g + 4 half of the panel
    __device__ __forceinline__ u32x4 read(uint32_t panel, int f, int half) const {
        if constexpr (!ACROSS) {
            const int rows = INTERLEAVED ? 64 * (f >> 2) + 4 * (f & 3) : 16 * f;
            return lds_read<u32x4>(panel + at[half] + rows * 128);
        } else if constexpr (SIZE == 2) {
            const uint32_t a = panel + at[f] + half * 32 * P::kPitch;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<HR_LDS s16x4 *>(a));
            const s16x4 hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<HR_LDS s16x4 *>(a + 4 * P::kPitch));
            const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
            return u32x4{l.x, l.y, h.x, h.y};
        } else {
            const uint32_t a = panel + at[f] + half * 64 * P::kPitch;
            const i32x2 l = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<HR_LDS i32x2 *>(a));
            const i32x2 h =
                __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<HR_LDS i32x2 *>(a + 8 * P::kPitch));
            return u32x4{static_cast<uint32_t>(l.x), static_cast<uint32_t>(l.y), static_cast<uint32_t>(h.x),
                         static_cast<uint32_t>(h.y)};
        }
    }
};

template <class E>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (__is_same(E, BF16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
}

// Four sums rounded once each to 16 bits.
template <class O>
__device__ __forceinline__ u32x2 narrow4(f32x4 v) {
    if constexpr (__is_same(O, BF16)) {
        const bf16x2 lo = {static_cast<__bf16>(v.x), static_cast<__bf16>(v.y)};
        const bf16x2 hi = {static_cast<__bf16>(v.z), static_cast<__bf16>(v.w)};
        return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    } else {
        const f16x2 lo = {static_cast<_Float16>(v.x), static_cast<_Float16>(v.y)};
        const f16x2 hi = {static_cast<_Float16>(v.z), static_cast<_Float16>(v.w)};
        return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    }
}

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
    return i32x8{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
                 static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
}

// (scales of 1: exponents of 127)
__device__ __forceinline__ f32x4 mfma8(i32x8 a, i32x8 b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0, 0, 0, 0}, 0, 0, 0, 0x7F7F7F7F, 0,
                                                            0x7F7F7F7F);
}

// A unit of a row at any address, of which `left` values (0 or fewer: none) are
// there; zeros for the others, whose memory is not touched.
template <int SIZE>
__device__ __forceinline__ u32x4 any_unit(const char *p, int left) {
    constexpr int UNIT = 16 / SIZE;
    u32x4 v = {0, 0, 0, 0};
    if (left >= UNIT) return load_vec<false>(p);
#pragma unroll
    for (int e = 0; e < UNIT - 1; ++e) {
        if (e < left) {
            const uint32_t x = SIZE == 2 ? *reinterpret_cast<const uint16_t *>(p + 2 * e)
                                         : *reinterpret_cast<const uint8_t *>(p + e);
            v[e * SIZE / 4] |= x << (8 * (e * SIZE % 4));
        }
    }
    return v;
}

// A unit's bytes moved down by `bytes` (0 .. 16), zeros behind them.
__device__ __forceinline__ u32x4 moved_down(u32x4 v, int bytes) {
    uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
    const int n = 8 * (bytes & 7);
    lo = n == 0 ? lo : lo >> n | hi << (64 - n);
    hi >>= n;
    if (bytes >= 8) lo = hi, hi = 0;
    if (bytes >= 16) lo = 0;
    return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                 static_cast<uint32_t>(hi >> 32)};
}

// Expert e's rows, whatever the offsets hold: inside 0 .. rows, first <= last.
__device__ __forceinline__ void segment(const int32_t *offsets, uint32_t all, int e, uint32_t &first, uint32_t &last) {
    if (offsets == nullptr) {
        first = 0;
        last = all;
        return;
    }
    const int lo = offsets[e], hi = offsets[e + 1], rows = static_cast<int>(all);
    first = lo < 0 ? 0 : lo > rows ? rows : lo;
    last = hi < static_cast<int>(first) ? first : hi > rows ? rows : hi;
}

struct Tile {
    bool there;
    int expert, q, p;                   // q, p: tile numbers
    uint32_t first, last;               // the expert's rows
};

// Consecutive workgroups go to the 8 dies in turn; each die takes a run of
// consecutive tiles, so that what its tiles share stays in its own cache.
//
// DEALT: runs of 16, and an eighth each of what is left, where tiles differ in time
// or take longer than their panels: the gradient of 2151 rows of 8 segments, 1327 x
// 1001, 39 -> 27 us, of 16384 of 32, 4097 x 4097, 1846 -> 1416, its product 1154 -> 1073;
// but the product of 64 matrices that are read for 32 rows each 176 -> 228.
template <bool DEALT>
__device__ __forceinline__ bool on_die(uint32_t group, uint32_t tiles, uint32_t &tile) {
    const uint32_t i = group / 8;
    uint32_t before = 0, run = (tiles + 7) / 8, at = i;
    if constexpr (DEALT) {
        constexpr uint32_t RUN = 16;
        before = i / RUN * (8 * RUN);
        if (before >= tiles) return false;
        run = tiles - before < 8 * RUN ? (tiles - before + 7) / 8 : RUN;
        at = i % RUN;
    }
    tile = before + group % 8 * run + at;
    return at < run && tile < tiles;
}

// Tile number t of nq x np: bands of 4 q, so that 32 running tiles are 4 x 8.
__device__ __forceinline__ void in_bands(uint32_t t, uint32_t nq, uint32_t np, int &q, int &p) {
    const uint32_t band = t / (4 * np), rest = t - band * 4 * np;
    const uint32_t high = nq - 4 * band < 4 ? nq - 4 * band : 4;
    p = static_cast<int>(rest / high);
    q = static_cast<int>(4 * band + rest % high);
}

// Which tile of the product this workgroup computes: the segments' tiles one
// after the other, counted by every wave for itself, 64 experts at a time.
template <int BQ, bool ANY>
__device__ __forceinline__ Tile product_tile(const ProductArgs &a, uint32_t group) {
    Tile t{};
    const int lane = threadIdx.x % kWave;
    uint32_t mine = 0;
    for (int e = lane; e < a.experts; e += kWave) {
        uint32_t lo, hi;
        segment(a.offsets, a.rows, e, lo, hi);
        mine += (hi - lo + BQ - 1) / BQ;
    }
    const uint32_t tiles = reduce_lanes<64>(mine, [](uint32_t x, uint32_t y) { return x + y; }) * a.tiles_p;
    uint32_t tile;
    t.there = on_die<ANY>(__builtin_amdgcn_readfirstlane(group), __builtin_amdgcn_readfirstlane(tiles), tile);
    if (!t.there) return t;
    for (int e0 = 0; e0 < a.experts; e0 += kWave) {
        uint32_t lo = 0, hi = 0;
        if (e0 + lane < a.experts) segment(a.offsets, a.rows, e0 + lane, lo, hi);
        const uint32_t n = (hi - lo + BQ - 1) / BQ * a.tiles_p;
        uint32_t upto = n;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const uint32_t v = __shfl_up(upto, d);
            if (lane >= d) upto += v;
        }
        const uint64_t past = __ballot(tile < upto);
        if (past != 0) {
            const int at = __builtin_ctzll(past);
            t.expert = __builtin_amdgcn_readfirstlane(e0 + at);
            t.first = __builtin_amdgcn_readlane(lo, at);
            t.last = __builtin_amdgcn_readlane(hi, at);
            const uint32_t all = __builtin_amdgcn_readlane(n, at), end = __builtin_amdgcn_readlane(upto, at);
            in_bands(tile - (end - all), all / a.tiles_p, a.tiles_p, t.q, t.p);
            return t;
        }
        tile -= __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    t.there = false;
    return t;
}

__device__ __forceinline__ Tile gradient_tile(const ProductArgs &a, uint32_t group) {
    Tile t{};
    const uint32_t each = static_cast<uint32_t>(a.tiles_q) * a.tiles_p;
    uint32_t tile;
    t.there = on_die<true>(group, each * a.experts, tile);
    if (!t.there) return t;
    t.expert = static_cast<int>(tile / each);
    in_bands(tile % each, a.tiles_q, a.tiles_p, t.q, t.p);
    uint32_t lo, hi;
    segment(a.offsets, a.rows, t.expert, lo, hi);
    t.first = __builtin_amdgcn_readfirstlane(lo);
    t.last = __builtin_amdgcn_readfirstlane(hi);
    return t;
}

template <class O>
constexpr int kOut = __is_same(O, float) ? 4 : 2;       // bytes

// The same value, of which the compiler knows nothing: what is computed from it
// is computed where it stands, and held in no register before.
__device__ __forceinline__ uint32_t here_only(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Registers f0 .. f3 of the lanes 16 g .. 16 g + 15 become registers g0 .. g3 of
// the lanes 16 f ..: a transposition of four registers and four groups of lanes.
__device__ __forceinline__ void exchange4(uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
    const auto ac = __builtin_amdgcn_permlane32_swap(a, c, false, false);
    const auto bd = __builtin_amdgcn_permlane32_swap(b, d, false, false);
    const auto ab = __builtin_amdgcn_permlane16_swap(ac[0], bd[0], false, false);
    const auto cd = __builtin_amdgcn_permlane16_swap(ac[1], bd[1], false, false);
    a = ab[0], b = ab[1], c = cd[0], d = cd[1];
}

// A wave's sums to the tile's rows at `out`: operand j of Q is its rows q_of(j) ..
// q_of(j) + 15, the wave's first value of P is p0; nq rows and np values are there.
// A lane holds row q_of(j) + lane % 16, and per operand of P four adjacent values:
// laced, 16 of four operands; in 16 bits made so (stores of 8 bytes to rows 32
// bytes long each are slower).
template <class O, bool LACED, bool NT, int FP, int FQ, class Q>
__device__ __forceinline__ void store_sums(const f32x4 (&sum)[FP][FQ], char *out, size_t stride, Q q_of, int p0, int nq,
                                           int np, uint32_t lane_) {
    const uint32_t lane = here_only(lane_);
    constexpr int OB = kOut<O>, RUN = LACED || (OB == 2 && FP % 4 == 0) ? 4 : 1;    // operands side by side
    const int g = lane >> 4;
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
        const int q = q_of(j) + (lane & 15);
        char *row = out + q * stride;
#pragma unroll
        for (int i = 0; i < FP; i += RUN) {
            const int p = p0 + 16 * i + (RUN == 4 ? 16 * g : 4 * g);
            if constexpr (OB == 4) {
                if (q >= nq) continue;
#pragma unroll
                for (int r = 0; r < RUN; ++r) {
                    if (p + 4 * r + 4 <= np) {
                        f32x4_row *to = reinterpret_cast<f32x4_row *>(row + (p + 4 * r) * 4);
                        if constexpr (NT)
                            __builtin_nontemporal_store(sum[i + r][j], to);
                        else
                            *to = sum[i + r][j];
                    } else {
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (p + 4 * r + v < np)
                                *reinterpret_cast<float *>(row + (p + 4 * r + v) * 4) = sum[i + r][j][v];
                    }
                }
            } else {
                u32x2 v[RUN];
#pragma unroll
                for (int r = 0; r < RUN; ++r) v[r] = narrow4<O>(sum[i + r][j]);
                if constexpr (RUN == 4 && !LACED) {
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) lo[r] = v[r].x, hi[r] = v[r].y;
                    exchange4(lo[0], lo[1], lo[2], lo[3]);
                    exchange4(hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = u32x2{lo[r], hi[r]};
                }
                if (q >= nq) continue;
                if (p + 4 * RUN <= np) {
                    if constexpr (RUN == 4) {
                        const u32x4 v0 = {v[0].x, v[0].y, v[1].x, v[1].y}, v1 = {v[2].x, v[2].y, v[3].x, v[3].y};
                        store_vec<NT>(v0, row + p * 2);
                        store_vec<NT>(v1, row + p * 2 + 16);
                    } else {
                        *reinterpret_cast<u32x2_row *>(row + p * 2) = v[0];
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < RUN; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (p + 4 * r + e < np)
                                *reinterpret_cast<uint16_t *>(row + (p + 4 * r + e) * 2) =
                                    static_cast<uint16_t>(v[r][e / 2] >> (16 * (e & 1)));
                }
            }
        }
    }
}

// A kernel's shape: tiles of BQ x BP; WQ x WP waves over them, WK times over
// the panels of a stage (each of which then takes its own panel); S stages.
template <int BQ_, int BP_, int WQ_, int WP_, int WK_, int S_, int GROUPS_ = 1>
struct Shape {
    static constexpr int BQ = BQ_, BP = BP_, WQ = WQ_, WP = WP_, WK = WK_, S = S_;
    static constexpr int kThreads = WQ * WP * WK * kWave;
    static constexpr int kMinWaves = WQ * WP * WK * GROUPS_ / 4 > 0 ? WQ * WP * WK * GROUPS_ / 4 : 1;   // a SIMD
};

// E: operands; O: out (F16, BF16 or float); QA, PA: the operand lies across.
// GRAD: the weights' gradient.  ANY: rows of any address and length, brought
// through registers.
//
// Waves that share a panel meet once a stage, after their loads of it have landed
// and before those of S - 1 stages later go out; a wave with a panel of its own
// (WK > 1) meets nobody until the sums are joined.  For few rows bound by HBM: 512
// rows of 64 matrices of 2560 x 5120 246 us (6.8 TB/s of weights), padded to 16 rows
// 254-264; e4m3 384 rows of 64 of 5120 x 5120 237 (7.1 TB/s); two rows of two
// matrices of 2048 x 4096 6.5 (a graph node alone 1.6).
template <class E, class O, class SH, bool QA, bool PA, bool GRAD, bool ANY>
__global__ __launch_bounds__(SH::kThreads, SH::kMinWaves) void product_tiles(ProductArgs a) {
    constexpr int SIZE = kBytes<E>, BQ = SH::BQ, BP = SH::BP, S = SH::S;
    constexpr int PQ = BQ / SH::WQ, PP = BP / SH::WP;           // a wave's part of the tile
    constexpr int FQ = PQ / 16, FP = PP / 16;
    constexpr bool LACED = !PA && PP % 64 == 0;                 // P's rows interleaved by four operands
    static_assert(PQ % 16 == 0 && PP % 16 == 0, "whole operands");
    using PanelQ = Panel<SIZE, BQ, QA, false>;
    using PanelP = Panel<SIZE, BP, PA, LACED>;
    constexpr int CK = PanelQ::kC;
    constexpr int kWaves = SH::WQ * SH::WP;                     // that share a panel
    constexpr bool SCALED = SIZE == 1;
    constexpr int kPanelBytes = PanelQ::kBytesAll + PanelP::kBytesAll + (SCALED ? BQ * 4 : 0);
    constexpr int kStageBytes = kPanelBytes * SH::WK;
    static_assert(PanelQ::kDmas % kWaves == 0 && PanelP::kDmas % kWaves == 0, "waves share a panel's loads evenly");
    constexpr int DQ = PanelQ::kDmas / kWaves, DP = PanelP::kDmas / kWaves;
    constexpr int kLoads = DQ + DP + (SCALED ? 1 : 0);          // a wave's, a stage
    static_assert(!SCALED || BQ / kWaves <= kWave, "a lane per scale");
    constexpr int kJoin = SH::WK > 1 ? (SH::WK - 1) * FQ * FP * 1024 * kWaves : 0;
    __shared__ __align__(1024) char lds[S * kStageBytes > kJoin ? S * kStageBytes : kJoin];

    const Tile tile = GRAD ? gradient_tile(a, blockIdx.x) : product_tile<BQ, ANY>(a, blockIdx.x);
    if (!tile.there) return;
    const uint32_t lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wk = wave / kWaves, share = wave % kWaves, wq = share % SH::WQ, wp = share / SH::WQ;

    // the tile's part of the operands
    const int q0 = tile.q * BQ, p0 = tile.p * BP;
    const int nq = GRAD ? a.nq - q0 : static_cast<int>(tile.last - tile.first) - q0;
    const int np = a.np - p0;
    const int nc = GRAD ? static_cast<int>(tile.last - tile.first) : a.nc;
    const int panels = (nc + CK - 1) / CK;
    const char *qs = a.q, *ps = a.p;
    if constexpr (GRAD) {
        qs += tile.first * a.q_stride + static_cast<size_t>(q0) * SIZE;
        ps += tile.first * a.p_stride + static_cast<size_t>(p0) * SIZE;
    } else {
        qs += (static_cast<size_t>(tile.first) + q0) * a.q_stride;
        ps += tile.expert * a.p_expert_stride + (PA ? static_cast<size_t>(p0) * SIZE : p0 * a.p_stride);
    }
    const size_t q_step = QA ? CK * a.q_stride : 128, p_step = PA ? CK * a.p_stride : 128;
    const float *xs = nullptr, *ws = nullptr;
    if constexpr (SCALED) {
        xs = a.q_scales + (static_cast<size_t>(tile.first) + q0) * a.q_scales_stride;
        // (a wave's part of p lies in one block of 128)
        const int block = (p0 + wp * PP) / 128, last = (a.np - 1) / 128;
        ws = a.p_scales + tile.expert * a.scales_expert + (block < last ? block : last) * a.scales_p;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(HR_LDS char *)lds;
    const uint32_t mine = lds0 + wk * kPanelBytes;              // this wave's panel of stage 0

    // the lanes' offsets of every load of a stage
    uint32_t off_q[DQ], off_p[DP], off_s = kNowhere;
#pragma unroll
    for (int j = 0; j < DQ; ++j) {
        uint32_t row, unit;
        PanelQ::source(share * DQ + j, lane, row, unit);
        off_q[j] = PanelQ::there(row, unit, nq, CK) ? static_cast<uint32_t>(row * a.q_stride) + unit * 16 : kNowhere;
    }
#pragma unroll
    for (int j = 0; j < DP; ++j) {
        uint32_t row, unit;
        PanelP::source(share * DP + j, lane, row, unit);
        off_p[j] = PanelP::there(row, unit, np, CK) ? static_cast<uint32_t>(row * a.p_stride) + unit * 16 : kNowhere;
    }
    constexpr int SROWS = BQ / kWaves;
    if constexpr (SCALED) {
        const int row = share * SROWS + lane;
        if (lane < SROWS && row < nq) off_s = static_cast<uint32_t>(row * a.q_scales_stride * 4);
    }

    // the loads of stage s (panels s * WK + wk), into buffer b
    const auto bring = [&](int s, int b) {
        const int panel = s * SH::WK + wk;
        const uint32_t to = mine + b * kStageBytes;
        const int left = nc - panel * CK;
        const i32x4 fq = buffer_of(qs + panel * q_step), fp = buffer_of(ps + panel * p_step);
        if (left >= CK) {
#pragma unroll
            for (int j = 0; j < DQ; ++j) dma16(fq, off_q[j], to + (share * DQ + j) * 1024);
#pragma unroll
            for (int j = 0; j < DP; ++j) dma16(fp, off_p[j], to + PanelQ::kBytesAll + (share * DP + j) * 1024);
        } else {
#pragma unroll
            for (int j = 0; j < DQ; ++j) {
                uint32_t row, unit;
                PanelQ::source(share * DQ + j, lane, row, unit);
                dma16(fq, PanelQ::there(row, unit, nq, left) ? off_q[j] : kNowhere, to + (share * DQ + j) * 1024);
            }
#pragma unroll
            for (int j = 0; j < DP; ++j) {
                uint32_t row, unit;
                PanelP::source(share * DP + j, lane, row, unit);
                dma16(fp, PanelP::there(row, unit, np, left) ? off_p[j] : kNowhere,
                      to + PanelQ::kBytesAll + (share * DP + j) * 1024);
            }
        }
        if constexpr (SCALED) {
            const i32x4 fs = buffer_of(reinterpret_cast<const char *>(xs + panel));
            if (lane < SROWS)
                dma4(fs, left > 0 ? off_s : kNowhere,
                     to + PanelQ::kBytesAll + PanelP::kBytesAll + share * SROWS * 4);
        }
    };

    Reader<SIZE, BQ, QA, false, FQ> from_q;
    Reader<SIZE, BP, PA, LACED, FP> from_p;
    from_q.init(wq * PQ, lane);
    from_p.init(wp * PP, lane);

    f32x4 sum[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) sum[i][j] = f32x4{0, 0, 0, 0};

    const int stages = (panels + SH::WK - 1) / SH::WK;
    // the sums over the panel at pq (stage s)
    const auto add = [&](int s, uint32_t pq) {
        const uint32_t pp = pq + PanelQ::kBytesAll;
        if constexpr (!SCALED) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                u32x4 x[FQ], w[FP];
#pragma unroll
                for (int j = 0; j < FQ; ++j) x[j] = from_q.read(pq, j, half);
#pragma unroll
                for (int i = 0; i < FP; ++i) w[i] = from_p.read(pp, i, half);
#pragma unroll
                for (int i = 0; i < FP; ++i)
#pragma unroll
                    for (int j = 0; j < FQ; ++j) sum[i][j] = mfma16<E>(w[i], x[j], sum[i][j]);
            }
        } else {
            const int panel = s * SH::WK + wk;
            const float block = panel < panels ? constant_at(ws + panel * a.scales_c) : 0.0f;
            i32x8 x[FQ];
            float scale[FQ];
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                x[j] = join(from_q.read(pq, j, 0), from_q.read(pq, j, 1));
                scale[j] = lds_read<float>(pp + PanelP::kBytesAll + (wq * PQ + 16 * j + (lane & 15)) * 4) * block;
            }
#pragma unroll
            for (int i = 0; i < FP; ++i) {
                const i32x8 w = join(from_p.read(pp, i, 0), from_p.read(pp, i, 1));
#pragma unroll
                for (int j = 0; j < FQ; ++j) {
                    const f32x4 part = mfma8(w, x[j]);
#pragma unroll
                    for (int v = 0; v < 4; ++v) sum[i][j][v] = fmaf(part[v], scale[j], sum[i][j][v]);
                }
            }
        }
    };

    if constexpr (!ANY) {
#pragma unroll
        for (int s = 0; s < S - 1; ++s)
            if (s < stages) bring(s, s);
        int b = 0;
        for (int s = 0; s < stages; ++s) {
            if (s + S - 2 < stages)
                landed<(S - 2) * kLoads>();
            else
                landed<0>();
            if constexpr (kWaves > 1) meet();
            if (s + S - 1 < stages) bring(s + S - 1, b == 0 ? S - 1 : b - 1);
            add(s, mine + b * kStageBytes);
            b = b == S - 1 ? 0 : b + 1;
        }
    } else {
        static_assert(S == 2, "one stage in registers");
        u32x4 in_q[DQ], in_p[DP];
        float in_s = 0.0f;
        // Whole units wherever a row has one: rows and units that are not there
        // are read from ones that are.  A unit that the row's end cuts is read so
        // that it ends there, and moved down when it goes to LDS; what lies past a
        // panel's c is made zero there, in the last panel alone and in those behind
        // it (a row or column of out that is not there may hold anything).  The loads are straight code: a
        // branch for every unit made each wait for the one before.
        constexpr int UNIT = PanelQ::kUnit;
        const bool narrow = (QA ? a.nq : nc) < UNIT || (PA ? a.np : nc) < UNIT;
        // unit d of a panel: its row, the values left of its row's from it on, and how
        // far before its place it is read
        const auto unit_of = [&](auto panel, bool across, int d, int b, int left, int &r, uint32_t &unit, int &here,
                                 int &back) {
            typedef decltype(panel) Pan;
            uint32_t row;
            Pan::source(share * (Pan::kDmas / kWaves) + d, lane, row, unit);
            const int wide = across ? b : left, u = static_cast<int>(unit) * UNIT;
            r = static_cast<int>(row);
            here = wide - u;
            back = here >= UNIT ? 0 : here > 0 ? UNIT - here : u + UNIT - wide;
        };
        const auto fetch_one = [&](auto panel, bool across, int d, const char *from, size_t stride, int b, int left) {
            int r, here, back;
            uint32_t unit;
            unit_of(panel, across, d, b, left, r, unit, here, back);
            const int rows = across ? left : b;
            return load_vec<false>(from + static_cast<size_t>(r < rows ? r : rows - 1) * stride +
                                   (static_cast<int>(unit) * 16 - back * SIZE));
        };
        const auto narrow_one = [&](auto panel, bool across, int d, const char *from, size_t stride, int b, int left) {
            int r, here, back;
            uint32_t unit;
            unit_of(panel, across, d, b, left, r, unit, here, back);
            return any_unit<SIZE>(from + r * stride + unit * 16, r < (across ? left : b) ? here : 0);
        };
        const auto trimmed = [&](auto panel, bool across, int d, u32x4 v, int b, int left) {
            int r, here, back;
            uint32_t unit;
            unit_of(panel, across, d, b, left, r, unit, here, back);
            v = moved_down(v, here >= UNIT ? 0 : here > 0 ? back * SIZE : 16);
            return across && r >= left ? u32x4{0, 0, 0, 0} : v;
        };
        const auto fetch = [&](int s) {
            const int panel = s * SH::WK + wk, left = nc - panel * CK;
            const char *fq = qs + panel * q_step, *fp = ps + panel * p_step;
            if (narrow) {
#pragma unroll
                for (int j = 0; j < DQ; ++j) in_q[j] = narrow_one(PanelQ(), QA, j, fq, a.q_stride, nq, left);
#pragma unroll
                for (int j = 0; j < DP; ++j) in_p[j] = narrow_one(PanelP(), PA, j, fp, a.p_stride, np, left);
            } else {
#pragma unroll
                for (int j = 0; j < DQ; ++j) in_q[j] = fetch_one(PanelQ(), QA, j, fq, a.q_stride, nq, left);
#pragma unroll
                for (int j = 0; j < DP; ++j) in_p[j] = fetch_one(PanelP(), PA, j, fp, a.p_stride, np, left);
            }
            if constexpr (SCALED)
                in_s = off_s != kNowhere && left > 0 ? xs[(share * SROWS + lane) * a.q_scales_stride + panel] : 0.0f;
        };
        const auto put = [&](int s) {
            const int left = nc - (s * SH::WK + wk) * CK;
            const uint32_t to = mine + (s & 1) * kStageBytes;
            if (!narrow && (left < CK || (QA && nq < BQ) || (PA && np < BP))) {
#pragma unroll
                for (int j = 0; j < DQ; ++j) in_q[j] = trimmed(PanelQ(), QA, j, in_q[j], nq, left);
#pragma unroll
                for (int j = 0; j < DP; ++j) in_p[j] = trimmed(PanelP(), PA, j, in_p[j], np, left);
            }
#pragma unroll
            for (int j = 0; j < DQ; ++j)
                *reinterpret_cast<HR_LDS u32x4 *>(to + (share * DQ + j) * 1024 + lane * 16) = in_q[j];
#pragma unroll
            for (int j = 0; j < DP; ++j)
                *reinterpret_cast<HR_LDS u32x4 *>(to + PanelQ::kBytesAll + (share * DP + j) * 1024 + lane * 16) = in_p[j];
            if (SCALED && lane < SROWS)
                *reinterpret_cast<HR_LDS float *>(to + PanelQ::kBytesAll + PanelP::kBytesAll + (share * SROWS + lane) * 4) =
                    in_s;
        };
        if (stages > 0) {
            fetch(0);
            put(0);
        }
        for (int s = 0; s < stages; ++s) {
            __syncthreads();
            if (s + 1 < stages) fetch(s + 1);
            add(s, mine + (s & 1) * kStageBytes);
            if (s + 1 < stages) put(s + 1);
        }
    }

    if constexpr (SH::WK > 1) {
        // the waves' sums over their panels, joined in order
        landed<0>();
        meet();
        const uint32_t at = lds0 + ((wk - 1) * kWaves + share) * FQ * FP * 1024 + lane * 16;
        if (wk > 0) {
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) *reinterpret_cast<HR_LDS f32x4 *>(at + (i * FQ + j) * 1024) = sum[i][j];
        }
        landed<0>();
        meet();
        if (wk > 0) return;
#pragma unroll
        for (int k = 0; k < SH::WK - 1; ++k)
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j)
                    sum[i][j] += lds_read<f32x4>(lds0 + (k * kWaves + share) * FQ * FP * 1024 + lane * 16 +
                                                 (i * FQ + j) * 1024);
    }

    char *out = a.out + (GRAD ? tile.expert * a.out_expert_stride + static_cast<size_t>(q0) * a.out_stride
                              : (static_cast<size_t>(tile.first) + q0) * a.out_stride);
    store_sums<O, LACED, false, FP, FQ>(sum, out + static_cast<size_t>(p0) * kOut<O>, a.out_stride,
                                 [&](int j) { return wq * PQ + 16 * j; }, wp * PP, nq, np, lane);
}

// The large tile: 256 x 256 by eight waves of 128 x 64, which read 24 KB of LDS
// for 64 matrix instructions and 64 KB of memory for 512.
//
// Two sets of four waves, one wave of each set on every SIMD, take turns: while
// one set's matrix instructions run, the other reads its operands, and a barrier
// changes them over.  A stage is one panel of P and two of Q (rows 0..127 and
// 128..255 of the tile; a wave has 64 of each), and is worked on in two turns,
// one for each panel of Q:
//
//     turn          4 s    4 s + 1   4 s + 2   4 s + 3   4 s + 4
//     first set     read   multiply  read      multiply  read
//     second set           read      multiply  read      multiply
//
// P and the first panel of Q were last read in turn 4 s + 1, the second panel in
// 4 s + 3.  So the loads of stage s + 2's P and first panel go out with the second
// reading of stage s, those of stage s + 1's second panel with the first; in 16
// bits behind the reads, in e4m3, where the reading turns are the longer ones,
// between the matrix instructions that follow (8192 x 8192 x 8192 520 -> 487 us; in
// 16 bits 749 behind the reads, 804 between).  A set waits for its own loads before
// the barrier after which either set reads them, four to six turns later.  Every
// turn of a wave issues the same number of loads, the last stages' from nowhere,
// so that the turns are straight code and the waits' counts fixed.
// A tile of at most 128 rows takes one turn per stage, and has three buffers.
//
// Tiles one after the other: a workgroup has a compute unit to itself.  The next
// tile's first loads go out before this one's sums are stored, and the stores
// are waited for a stage later (loads and stores complete in order).
//
// 8192 x 8192 x 8192, normally distributed values: bfloat16 730-760 us (1.45-1.51 PF),
// transposed 753, gradient 760-787; e4m3 465-488 (2.3 PF; 500-540 where every 97th
// value is 8 times as large).  Without any loads bfloat16 and e4m3 take 640 and 411,
// with zeros for data e4m3 takes 400 with loads: the rest is power.  Instructions of 32
// x 32 x 16 instead of 16 x 16 x 32: 812 against 760.  The next tile's loads and the
// sets' turns without a break between tiles: 787 against 762.  Segments of 512 rows of
// 128 matrices (4096 -> 2048) 895: a die's 32 tiles have 20 panels there, of one large
// matrix 12.
template <class E, class O, bool QA, bool PA, bool GRAD>
__global__ __launch_bounds__(512, 2) void product_large(ProductArgs a) {
    constexpr int SIZE = kBytes<E>, BQ = 256, BP = 256, H = 128, FP = 4, FH = 4;
    constexpr bool LACED = !PA, SCALED = SIZE == 1;
    using PanelQ = Panel<SIZE, H, QA, false>;
    using PanelP = Panel<SIZE, BP, PA, LACED>;
    constexpr int CK = PanelP::kC;
    constexpr uint32_t QB = PanelQ::kBytesAll, PB = PanelP::kBytesAll;      // 16 and 32 KB
    constexpr uint32_t kScales = 3 * (PB + QB), kTable = kScales + (SCALED ? 4 * BQ * 4 : 0);
    constexpr int D0 = 6 + SCALED, D1 = 2;                                  // a wave's loads for the turns
    constexpr int STORES = kOut<O> == 4 ? FP * FH : FH * 2;                 // of a wave and turn, full tile
    // (and the segments' first rows, and their tiles counted up, or their order)
    __shared__ __align__(1024) char lds[kTable + (2 * HR_EXPERTS_MAX + 1) * 4];

    const uint32_t lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const bool second = wave >= 4;
    const int wq = wave & 1, wp = wave >> 1;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(HR_LDS char *)lds;
    const uint32_t firsts = lds0 + kTable, counts = firsts + (HR_EXPERTS_MAX + 1) * 4;

    // the arguments, read again where a tile begins: they would fill the scalar
    // registers all the time
    typedef const __attribute__((address_space(4))) ProductArgs Arguments;
    const auto args = [] {
        Arguments *p = (Arguments *)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(p));
        return p;
    };
    for (int e = threadIdx.x; e <= a.experts; e += 512) {
        const int at = a.offsets != nullptr ? a.offsets[e] : e == 0 ? 0 : static_cast<int>(a.rows);
        const int rows = static_cast<int>(a.rows);
        *reinterpret_cast<HR_LDS int *>(firsts + e * 4) = at < 0 ? 0 : at > rows ? rows : at;
    }
    __syncthreads();
    uint32_t tiles;
    if constexpr (GRAD) {
        // The longest segments first, so that a round's tiles are alike, and every second
        // round the other way round (32 segments of 32768 rows, 1024 x 2048 199 -> 160
        // us, 1024 x 1024 112 -> 101).
        for (int e = threadIdx.x; e < a.experts; e += 512) {
            const int rows = lds_read<int>(firsts + e * 4 + 4) - lds_read<int>(firsts + e * 4);
            int longer = 0, lo = lds_read<int>(firsts);
#pragma unroll 8
            for (int i = 0; i < a.experts; ++i) {
                const int hi = lds_read<int>(firsts + i * 4 + 4);
                longer += hi - lo > rows || (hi - lo == rows && i < e);
                lo = hi;
            }
            *reinterpret_cast<HR_LDS int *>(counts + longer * 4) = e;
        }
        __syncthreads();
        tiles = static_cast<uint32_t>(a.tiles_q) * a.tiles_p * a.experts;
    } else {
        if (wave == 0) {
            uint32_t before = 0;
            for (int e = lane; e - static_cast<int>(lane) < a.experts; e += kWave) {
                uint32_t n = 0;
                if (e < a.experts) {
                    const int lo = lds_read<int>(firsts + e * 4), hi = lds_read<int>(firsts + e * 4 + 4);
                    n = hi > lo ? (hi - lo + BQ - 1) / BQ * a.tiles_p : 0;
                }
#pragma unroll
                for (int d = 1; d < kWave; d *= 2) {
                    const uint32_t v = __shfl_up(n, d);
                    if (static_cast<int>(lane) >= d) n += v;
                }
                if (e < a.experts) *reinterpret_cast<HR_LDS uint32_t *>(counts + e * 4) = before + n;
                before += __builtin_amdgcn_readlane(n, kWave - 1);
            }
        }
        __syncthreads();
        tiles = __builtin_amdgcn_readfirstlane(lds_read<uint32_t>(counts + (a.experts - 1) * 4));
    }
    // Rounds of a tile for every workgroup, an eighth of it for each die: a run, which
    // shares panels.  (With one run of all rounds' tiles for each die, one of them had
    // 1.5 to 1.8 times the work of the gradient of 32 segments: 16384 rows padded to
    // 128, 4096 x 4096, 772 -> 711 us, 696 with the longest first; 65528 rows of 128
    // experts, 4096 -> 2048, 1138 -> 1108.)  The product's places in a round move on by one every second round, so that
    // tiles of half the work (each second, third or fourth one of an expert) come to
    // all workgroups (384 rows for each of 128 experts, 4096 -> 2048: 892 -> 822, now 791).
    const uint32_t places = gridDim.x / 8, die = blockIdx.x % 8;
    uint32_t round = 0, t;
    const auto there = [&] {
        const uint32_t left = tiles - round * gridDim.x;
        const uint32_t run = left < gridDim.x ? (left + 7) / 8 : places;
        const uint32_t at = (blockIdx.x / 8 + (GRAD ? 0 : round / 2)) % places, deal = die * run + at;
        t = round * gridDim.x + (GRAD && round % 2 != 0 ? 8 * run - 1 - deal : deal);
        return round * gridDim.x < tiles && at < run && t < tiles;
    };
    if (!there()) return;

    // the tile's place: its part of the operands, of out, and what is there of it
    const char *qs, *ps;
    char *out;
    const float *xs = nullptr, *ws = nullptr;
    int nq, np, nc, stages;
    const size_t q_step = QA ? CK * a.q_stride : 128, p_step = PA ? CK * a.p_stride : 128;
    uint32_t off_p[4], off_q[4], off_s = kNowhere;
    int e0 = 0;                         // experts before have no tile left
    // offsets of a wave's loads: P, and the two panels of Q (c values of the stage
    // left; the last stage's are trimmed before its loads go out)
    const auto offsets = [&](int c) {
        const uint32_t l = here_only(lane);
        const auto &a = *args();
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t row, unit;
            PanelP::source(wave * 4 + d, l, row, unit);
            off_p[d] = PanelP::there(row, unit, np, c) ? static_cast<uint32_t>(row * a.p_stride) + unit * 16 : kNowhere;
            PanelQ::source(wave * 2 + (d & 1), l, row, unit);
            if constexpr (QA)
                unit += (d >> 1) * H / PanelQ::kUnit;
            else
                row += (d >> 1) * H;
            off_q[d] = PanelQ::there(row, unit, nq, c) ? static_cast<uint32_t>(row * a.q_stride) + unit * 16 : kNowhere;
        }
    };
    const auto place = [&] {
        const auto &a = *args();
        int expert, tq, tp;
        uint32_t first, last;
        if constexpr (GRAD) {
            const uint32_t per = static_cast<uint32_t>(a.tiles_q) * a.tiles_p;
            expert = __builtin_amdgcn_readfirstlane(lds_read<int>(counts + t / per * 4));
            in_bands(t % per, a.tiles_q, a.tiles_p, tq, tp);
            const int lo = __builtin_amdgcn_readfirstlane(lds_read<int>(firsts + expert * 4));
            const int hi = __builtin_amdgcn_readfirstlane(lds_read<int>(firsts + expert * 4 + 4));
            first = lo, last = hi < lo ? lo : hi;
        } else {
            uint32_t upto;
            uint64_t past;
            for (;; e0 += kWave) {
                // (the last count is past every tile)
                const int e = e0 + static_cast<int>(lane) < a.experts ? e0 + static_cast<int>(lane) : a.experts - 1;
                upto = lds_read<uint32_t>(counts + e * 4);
                past = __ballot(t < upto);
                if (past != 0) break;
            }
            expert = __builtin_amdgcn_readfirstlane(e0 + __builtin_ctzll(past));
            const int lo = __builtin_amdgcn_readfirstlane(lds_read<int>(firsts + expert * 4));
            const int hi = __builtin_amdgcn_readfirstlane(lds_read<int>(firsts + expert * 4 + 4));
            first = lo, last = hi;
            const uint32_t high = (last - first + BQ - 1) / BQ;
            const uint32_t all = __builtin_amdgcn_readfirstlane(lds_read<uint32_t>(counts + expert * 4));
            in_bands(t - (all - high * a.tiles_p), high, a.tiles_p, tq, tp);
        }
        const int q0 = tq * BQ, p0 = tp * BP;
        nq = GRAD ? a.nq - q0 : static_cast<int>(last - first) - q0;
        np = a.np - p0;
        nc = GRAD ? static_cast<int>(last - first) : a.nc;
        stages = (nc + CK - 1) / CK;
        if constexpr (GRAD) {
            qs = a.q + first * a.q_stride + static_cast<size_t>(q0) * SIZE;
            ps = a.p + first * a.p_stride + static_cast<size_t>(p0) * SIZE;
            out = a.out + expert * a.out_expert_stride + static_cast<size_t>(q0) * a.out_stride;
        } else {
            qs = a.q + (static_cast<size_t>(first) + q0) * a.q_stride;
            ps = a.p + expert * a.p_expert_stride + (PA ? static_cast<size_t>(p0) * SIZE : p0 * a.p_stride);
            out = a.out + (static_cast<size_t>(first) + q0) * a.out_stride;
        }
        out += static_cast<size_t>(p0) * kOut<O>;
        offsets(nc < CK ? nc : CK);
        if constexpr (SCALED) {
            xs = a.q_scales + (static_cast<size_t>(first) + q0) * a.q_scales_stride;
            const int block = (p0 + wp * 64) / 128, most = (a.np - 1) / 128;
            ws = a.p_scales + expert * a.scales_expert + (block < most ? block : most) * a.scales_p;
            const int row = wave % 4 * 64 + lane;               // (either set brings them all)
            off_s = row < nq ? static_cast<uint32_t>(row * a.q_scales_stride * 4) : kNowhere;
        }
    };
    const auto trim = [&](int s) {
        if (s == stages - 1 && s > 0 && nc % CK != 0) offsets(nc % CK);
    };
    // load d of a wave for the first turn of stage s, into buffer b, and for the
    // second
    const auto bring0 = [&](int s, int b, int d) {
        const bool here = s < stages;
        if (d < 4)
            dma16(buffer_of(ps + s * p_step, here), off_p[d], lds0 + b * PB + (wave * 4 + d) * 1024);
        else if (d < 6)
            dma16(buffer_of(qs + s * q_step, here), off_q[d - 4], lds0 + 3 * PB + b * QB + (wave * 2 + d - 4) * 1024);
        else
            dma4(buffer_of(reinterpret_cast<const char *>(xs + s), here), off_s,
                 lds0 + kScales + (s & 3) * BQ * 4 + wave % 4 * 256);
    };
    const auto bring1 = [&](int s, int b, int d) {
        dma16(buffer_of(qs + s * q_step, s < stages), off_q[2 + d], lds0 + 2 * PB + b * QB + (wave * 2 + d) * 1024);
    };

    Reader<SIZE, H, QA, false, FH> from_q;
    Reader<SIZE, BP, PA, LACED, FP> from_p;
    from_q.init(wq * 64, lane);
    from_p.init(wp * 64, lane);

    u32x4 w[2][FP], x[2][FH];
    i32x8 w8[FP], x8[FH];                                       // (e4m3: both halves as one operand)
    float block = 0.0f, scale[FH];
    const auto block_of = [&](int s) { block = constant_at(ws + (s < stages ? s : 0) * a.scales_c); };
    const auto read_p = [&](uint32_t at) {
#pragma unroll
        for (int i = 0; i < FP; ++i) {
            if constexpr (SCALED) {
                w8[i] = join(from_p.read(at, i, 0), from_p.read(at, i, 1));
            } else {
                w[0][i] = from_p.read(at, i, 0);
                w[1][i] = from_p.read(at, i, 1);
            }
        }
    };
    const auto read_q = [&](int s, int turn, uint32_t at) {
#pragma unroll
        for (int j = 0; j < FH; ++j) {
            if constexpr (SCALED) {
                x8[j] = join(from_q.read(at, j, 0), from_q.read(at, j, 1));
                scale[j] = lds_read<float>(lds0 + kScales + (s & 3) * BQ * 4 +
                                           (turn * H + wq * 64 + 16 * j + (lane & 15)) * 4) * block;
            } else {
                x[0][j] = from_q.read(at, j, 0);
                x[1][j] = from_q.read(at, j, 1);
            }
        }
    };
    // a turn's instructions for one panel of Q; e4m3: with the turn's loads between them
    const auto multiply = [&](f32x4 (&sum)[FP][FH], auto loads_, auto load) {
        constexpr int loads = decltype(loads_)::value;
        __builtin_amdgcn_s_setprio(1);
        if constexpr (!SCALED) {
#pragma unroll
            for (int t = 0; t < 2 * FP * FH; ++t) {
                const int half = t / (FP * FH), j = t / FP % FH, i = t % FP;
                sum[i][j] = mfma16<E>(w[half][i], x[half][j], sum[i][j]);
            }
        } else {
            // (a part is scaled four instructions later, when it is there: two later
            // the compiler put waits of up to 9 slots before every other scaling)
            constexpr int N = FP * FH, EACH = N / (loads + 1), LATER = 4;
            f32x4 part[LATER + 1];
#pragma unroll
            for (int t = 0; t < N + LATER; ++t) {
                if (t < N) part[t % (LATER + 1)] = mfma8(w8[t % FP], x8[t / FP]);
                __builtin_amdgcn_sched_barrier(0);
                if (t >= LATER) {
                    const int u = t - LATER;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        sum[u % FP][u / FP][v] =
                            fmaf(part[u % (LATER + 1)][v], scale[u / FP], sum[u % FP][u / FP][v]);
                }
                if (t % EACH == EACH - 1 && t / EACH < loads) load(t / EACH);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // (the sums are made here: the compiler would move them past the barriers)
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int j = 0; j < FH; ++j) asm volatile("" : "+v"(sum[i][j]));
        __builtin_amdgcn_s_setprio(0);
    };
    const auto clear = [](f32x4 (&sum)[FP][FH]) {
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int j = 0; j < FH; ++j) sum[i][j] = f32x4{0, 0, 0, 0};
    };
    // 16 bits: a turn's loads go out after its reads
    const auto reading = [&](auto loads_, auto load) {
        if constexpr (!SCALED) {
#pragma unroll
            for (int d = 0; d < decltype(loads_)::value; ++d) load(d);
        }
    };
    const std::integral_constant<int, D0> d0;
    const std::integral_constant<int, D1> d1;
    // the loads before a tile's first turns
    const auto begin = [&] {
        if constexpr (SCALED) block_of(0);
#pragma unroll
        for (int d = 0; d < D0; ++d) bring0(0, 0, d);
        if (nq > H) {
#pragma unroll
            for (int d = 0; d < D1; ++d) bring1(0, 0, d);
        }
        trim(1);
#pragma unroll
        for (int d = 0; d < D0; ++d) bring0(1, 1, d);
    };

    f32x4 sum0[FP][FH], sum1[FP][FH];
    place();
    begin();
    int stored = 0;                     // stores that are behind the first loads
    for (;;) {
        // all but the last n loads, and the last tile's stores, which a wave issued
        // after its first loads
        const auto wait = [&](auto n_, int s) {
            constexpr int n = decltype(n_)::value;
            if (s > 0 || stored == 0)
                landed<n>();
            else if (stored == STORES)
                landed<n + STORES>();
            else
                landed<n + 2 * STORES>();
        };
        clear(sum0);
        if (nq > H) {
            clear(sum1);
            wait(std::integral_constant<int, D0 + D1>(), 0);    // stage 0, for its first turn
            change();
            if (second) change();
            for (int s = 0; s < stages; ++s) {
                const int b = s & 1;
                read_p(lds0 + b * PB);
                read_q(s, 0, lds0 + 3 * PB + b * QB);
                const auto last = [&](int d) { bring1(s + 1, b ^ 1, d); };
                reading(d1, last);
                if (second) wait(std::integral_constant<int, SCALED ? D0 : D0 + D1>(), s);  // stage s, second turn
                read_done();
                change();
                multiply(sum0, d1, last);
                if (!second) wait(std::integral_constant<int, D0 + D1>(), s);               // the same
                change();
                read_q(s, 1, lds0 + 2 * PB + b * QB);
                trim(s + 2);
                const auto first = [&](int d) { bring0(s + 2, b, d); };
                reading(d0, first);
                if (second) wait(std::integral_constant<int, SCALED ? D1 : D0 + D1>(), s);  // stage s + 1, first turn
                read_done();
                change();
                if constexpr (SCALED) block_of(s + 1);
                multiply(sum1, d0, first);
                if (!second) wait(std::integral_constant<int, D0 + D1>(), s);               // the same
                change();
            }
            if (!second) change();
        } else {
            //     turn          2 s    2 s + 1   2 s + 2   2 s + 3
            //     first set     read   multiply  read      multiply
            //     second set           read      multiply  read
            wait(d0, 0);
            change();
            if (second) change();
            int b = 0;
            for (int s = 0; s < stages; ++s) {
                read_p(lds0 + b * PB);
                read_q(s, 0, lds0 + 3 * PB + b * QB);
                trim(s + 2);
                const int to = b == 0 ? 2 : b - 1;
                const auto first = [&](int d) { bring0(s + 2, to, d); };
                reading(d0, first);
                if (second) wait(std::integral_constant<int, SCALED ? 0 : D0>(), s);        // stage s + 1
                read_done();
                change();
                if constexpr (SCALED) block_of(s + 1);
                multiply(sum0, d0, first);
                if (!second) wait(d0, s);                                                   // stage s + 1
                change();
                b = b == 2 ? 0 : b + 1;
            }
            if (!second) change();
        }
        landed<0>();        // (loads from nowhere; after the last tile this LDS is another's)
        char *const to = out;
        const int rows = nq, width = np;
        ++round;
        const bool more = there();
        if (more) {
            place();
            begin();
        }
        const size_t out_stride = args()->out_stride;
        const auto store = [&](auto nt) {
            constexpr bool NT = decltype(nt)::value;
            store_sums<O, LACED, NT, FP, FH>(sum0, to, out_stride, [&](int j) { return wq * 64 + 16 * j; }, wp * 64, rows,
                                             width, lane);
            if (rows > H)
                store_sums<O, LACED, NT, FP, FH>(sum1, to, out_stride, [&](int j) { return H + wq * 64 + 16 * j; },
                                                 wp * 64, rows, width, lane);
        };
        if (GRAD && args()->stream)
            store(std::integral_constant<bool, GRAD>());
        else
            store(std::false_type());
        if (!more) break;
        // a partial tile's stores are not counted, but waited for
        stored = width >= BP && (rows == H || rows >= BQ) ? (rows > H ? 2 * STORES : STORES) : 0;
        if (stored == 0) landed<0>();
    }
}

}  // namespace hr
