// m3_attend_common.h -- what the two attention kernels share (m3_kv_attend.hip: few
// rows a sequence; m3_kv_attend_tile.hip: many). Device code only.
#pragma once
#include "m3_attn_device.h"
#include "m3_attn_internal.h"

namespace m3 {

// The kernels' forms: kPlain, without sinks and prefixes; kView, with them in one pass over
// each sequence's keys; kParts, one part over a group's prefix for all its rows (a sequence
// of keys like any other, whose rows are those of several sequences), one over each
// sequence's own keys, brought together afterwards.
enum Form { kPlain, kView, kParts };

// A call as the kernels take it.
struct AttendDev {
    m3_kv_cache c;
    m3_kv_batch b;
    m3_rows q;
    void* out;
    float* lse;
    // Parts of rows whose keys several workgroups share: the sums [..][D] in the part's
    // unit, and (log2 of the unit, the probabilities' sum) [..][2]. By [split][token]
    // [head], or with even shares by [slot][row of the tile] (m3_kv_attend.hip).
    float* part_o;
    float* part_ml;
    int* shares;     // even shares: tiles of a share, then the items' first tiles [items + 1]
    int items;       // (sequence, row tile) pairs; 0: no even shares
    int packed;      // log2 of `rows` where the pairs follow one another (unit_of), else 0
    int q_heads, group, D, shift, rows;
    float scale2;    // scale * log2(e)
    int causal;
    int64_t window, row_tiles, split_tiles;  // split_tiles: of a split, as far as the bound tells
    int splits;
    bool wide;
    int64_t blocks;  // workgroups with work (the grid may hold a few more)
    Form form;
    m3_kv_view view;
    int most_prefix;  // pages that a prefix may have: of a row of its table, ending within 32 bits
    // The kParts form: the groups' (group, row tile) pairs come before the sequences' among the
    // items, numbered by their own row tiles; where parts lie (in rows of part_o, part_ml).
    int items_a, packed_a, splits_a;  // splits_a: the prefix's parts by [split][token][head]; 0: even shares too
    int64_t row_tiles_a, slots, solo_a, solo_b;
    // of the tile kernel's launch:
    int columns;     // (sequence, head, split)s side by side in an XCD (0: runs of workgroups)
    int64_t grid;
};

hipError_t launch_attend_tile(const AttendDev& d, m3_dtype io, hipStream_t s);
// the other forms' instances (m3_kv_attend_view.hip, m3_kv_attend_parts.hip, m3_kv_attend_tile_view.hip)
hipError_t launch_rows_view(const AttendDev& d, m3_dtype io, hipStream_t s);
hipError_t launch_rows_parts(const AttendDev& d, m3_dtype io, hipStream_t s);
hipError_t launch_attend_tile_view(const AttendDev& d, m3_dtype io, hipStream_t s);
// Joins a prefix's parts with those of the sequences' own keys, where both are of even shares or
// the own ones are.
hipError_t launch_merge(const AttendDev& d, m3_dtype io, hipStream_t s);

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
constexpr float kF16Top = 32768.f;  // probabilities stay below it, in fp16's range
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;  // keys of a tile

__device__ __forceinline__ floatx4 mfma_f16(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}
__device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// The sequence and row tile of pair e, and back.
__device__ __forceinline__ Unit pair_of(const AttendDev& a, int e) {
    if (a.packed) return unit_of(a.b, e, a.group, a.packed, 1);
    return Unit{unsigned(e) / unsigned(a.row_tiles), unsigned(e) % unsigned(a.row_tiles)};
}
__device__ __forceinline__ int64_t pair_at(const AttendDev& a, int64_t i, int64_t rt) {
    return a.packed ? first_unit(a.b, i, a.group, a.packed, 1) + rt : i * a.row_tiles + rt;
}

// The group of sequence i (-1: none), and the pages that its sequences hold together.
__device__ __forceinline__ int64_t group_of(const AttendDev& a, int64_t i) {
    const m3_kv_view& v = a.view;
    if (v.groups == 0) return -1;
    int64_t g = 0;
    if (v.group_start) {  // the last group that begins at or before i
        for (int64_t hi = v.groups - 1; g < hi;) {
            const int64_t mid = (g + hi + 1) / 2;
            if (v.group_start[mid] <= i) g = mid;
            else hi = mid - 1;
        }
        if (i < v.group_start[g] || i >= v.group_start[g + 1]) return -1;
    }
    return g;
}
struct Prefix {
    const int32_t* pages;
    int count;
};
__device__ __forceinline__ Prefix prefix_at(const AttendDev& a, int64_t g) {
    const m3_kv_view& v = a.view;
    if (g < 0) return Prefix{nullptr, 0};
    return Prefix{v.prefix_pages + g * v.max_prefix, min(max(v.prefix_count[g], 0), a.most_prefix)};
}
__device__ __forceinline__ Prefix prefix_of(const AttendDev& a, int64_t i) { return prefix_at(a, group_of(a, i)); }

// A group's sequences and rows.
__device__ __forceinline__ int64_t sequence_at(const AttendDev& a, int64_t g) {  // its first (of g = groups: the end)
    const m3_kv_view& v = a.view;
    return v.group_start ? min(max(int64_t(v.group_start[g]), int64_t(0)), a.b.batch) : g * a.b.batch;
}
__device__ __forceinline__ int64_t row_at(const AttendDev& a, int64_t i) {  // a sequence's first row
    return a.b.cu_q ? min(max(int64_t(a.b.cu_q[i]), int64_t(0)), a.b.tokens) : i;
}
struct Group {
    int64_t first, last;  // its sequences (last: one beyond)
    int64_t row0;
    int n;                // rows
    int held;             // keys of its prefix
    Prefix pre;
};
__device__ __forceinline__ Group group_at(const AttendDev& a, int64_t g) {
    Group r;
    r.first = sequence_at(a, g);
    r.last = max(sequence_at(a, g + 1), r.first);
    r.row0 = row_at(a, r.first);
    r.n = int(max(row_at(a, r.last) - r.row0, int64_t(0)));
    r.pre = prefix_at(a, g);
    r.held = int(min(int64_t(r.pre.count) * a.c.page_size, a.b.max_kv));
    return r;
}
// Keys of its group's prefix that row `tok` sees: all, but where its sequence ends or (causal) it
// lies within.
__device__ __forceinline__ int row_limit(const AttendDev& a, const Group& gr, int64_t tok) {
    int64_t i = tok;
    if (a.b.cu_q) {  // the last sequence that begins at or before the row
        i = gr.first;
        for (int64_t hi = gr.last - 1; i < hi;) {
            const int64_t mid = (i + hi + 1) / 2;
            if (a.b.cu_q[mid] <= tok) i = mid;
            else hi = mid - 1;
        }
    }
    const Seq s = seq_of(a.b, i);
    const int64_t t = tok - s.row0;
    if (t < 0 || t >= s.n) return 0;
    int64_t hi = min(gr.held, s.held);
    if (a.causal) hi = min(hi, s.base + t + 1);
    return int(max(hi, int64_t(0)));
}
// The group and row tile of pair e, and back (as pair_of and pair_at).
__device__ __forceinline__ int64_t group_unit(const AttendDev& a, int64_t g) {
    return (row_at(a, sequence_at(a, g)) * a.group >> a.packed_a) + g;
}
__device__ __forceinline__ Unit group_pair_of(const AttendDev& a, int e) {
    if (!a.packed_a) return Unit{unsigned(e) / unsigned(a.row_tiles_a), unsigned(e) % unsigned(a.row_tiles_a)};
    int64_t g = 0;
    for (int64_t hi = a.view.groups - 1; g < hi;) {
        const int64_t mid = (g + hi + 1) / 2;
        if (group_unit(a, mid) <= e) g = mid;
        else hi = mid - 1;
    }
    return Unit{g, e - group_unit(a, g)};
}
__device__ __forceinline__ int64_t group_pair_at(const AttendDev& a, int64_t g, int64_t rt) {
    return a.packed_a ? group_unit(a, g) + rt : g * a.row_tiles_a + rt;
}

// Tiles of 64 keys that rows r0 .. r0 + rows - 1 of a sequence can see: number t of lo .. hi
// - 1 is tile t; in the kView form tile t + skip from the first that the window shows on.
struct Span {
    int64_t lo, hi;
    int sinks, skip;  // (kView) tiles of the sinks alone, tiles between them and the window's
};
// Keeps what is computed from a register after this point, where the compiler would form it
// early and hold it.
__device__ __forceinline__ unsigned here(unsigned w) {
    asm volatile("" : "+v"(w));
    return w;
}
template <Form F>
__device__ __forceinline__ int tile_at(const Span& sp, int t) {
    if constexpr (F == kView) return t < sp.sinks ? t : t + sp.skip;
    else return t;
}
template <Form F>
__device__ __forceinline__ Span span_of(const AttendDev& a, const Seq& s, int r0, int own = 0) {
    const int r1 = min(r0 + a.rows, s.n * a.group) - 1;
    const int64_t base = s.base;
    int64_t hi = min(int64_t(s.held), a.b.max_kv), lo = 0;
    if (a.causal) hi = min(hi, base + r1 / a.group + 1);
    if (a.window) lo = max(int64_t(0), base + r0 / a.group - a.window + 1);
    if constexpr (F == kParts) lo = own;  // (no window there; own: the sequence's first key of its own)
    if constexpr (F == kView) {
        const int64_t first = min(min(a.view.sinks, lo), hi);  // keys that only sinks show
        if (hi <= lo && first <= 0) return Span{0, 0, 0, 0};
        const int sinks = int((max(first, int64_t(0)) + kTile - 1) / kTile);
        if (hi <= lo) return Span{0, sinks, sinks, 0};
        const int from = int(lo / kTile), to = int((hi + kTile - 1) / kTile);
        const int skip = max(from - sinks, 0);
        return Span{0, to - skip, sinks, skip};
    } else {
        if (hi <= lo) return Span{0, 0, 0, 0};
        return Span{lo / kTile, (hi + kTile - 1) / kTile, 0, 0};
    }
}

// How the kernel for many rows cuts a row tile's keys: into as many pieces as the plan has
// workgroups for, from the keys that the tile sees (the plan knows a bound of them only),
// at least kPieceTiles tiles each. One piece is written out directly, parts are joined.
struct Cut {
    int per, pieces;
};
__device__ __forceinline__ Cut cut_of(int n, int splits, int least) {
    const int per = max((n + splits - 1) / splits, least);
    return Cut{per, max((n + per - 1) / per, 1)};
}
__device__ __forceinline__ Cut cut_of(const AttendDev& a, const Span& sp) {
    return cut_of(int(sp.hi - sp.lo), a.splits, kPieceTiles);
}

// 8 entries of a query row as MFMA operands: one bf16 part, or three that add
// up to the fp32 value.
template <typename T>
struct Parts;
template <>
struct Parts<bf16_t> {
    static constexpr int kN = 1;  // parts of a query
    static constexpr int kV = 1;  // parts of a probability
    __device__ __forceinline__ static void load(const bf16_t* p, bool wide, u32x4* f) {
        if (wide) {
            f[0] = *reinterpret_cast<const u32x4*>(p);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[0][j] = unsigned(p[2 * j].bits) | unsigned(p[2 * j + 1].bits) << 16;
        }
    }
};
__device__ __forceinline__ void split3(float lo, float hi, unsigned* w) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        w[k] = pack_bf16(lo, hi);
        lo -= __uint_as_float(w[k] << 16);
        hi -= __uint_as_float(w[k] & 0xffff0000u);
    }
}
template <>
struct Parts<float> {
    static constexpr int kN = 3;
    static constexpr int kV = 3;
    __device__ __forceinline__ static void load(const float* p, bool wide, u32x4* f) {
        float v[8];
        if (wide)
            load8<true>(p, v);
        else
            load8<false>(p, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            unsigned w[3];
            split3(v[2 * j], v[2 * j + 1], w);
#pragma unroll
            for (int k = 0; k < 3; ++k) f[k][j] = w[k];
        }
    }
};

// Probabilities. p' = 2^(s + log2 vs - M + kUp): the score s (log2), the scale vs of
// the key's V block, and the row's running reference M >= s + log2 vs - 8 of all keys
// so far, so that sum p' code is the output's numerator and sum p' / vs its
// denominator, in units of 2^(M - kUp). p' is at most 2^15. For the product with V bf16
// rows round it to fp16: 11 bits where bf16 would have 8, down to 2^-14 of the unit; below
// it the last of the bits is 2^-24, that is 2^-31 of a largest p' of 2^7. fp32 rows split it
// into three bf16 parts, which keep its 24 bits wherever it lies. The denominator takes p'
// in fp32, times 1 / vs of its block.
// A block whose scale is 0 (or below the normal numbers) holds zeros, whatever its
// codes: it counts as 2^-60.
constexpr float kUp = 7.f, kSlack = 8.f;
struct VScale {
    float log2, inv;
    bool none;
};
__device__ __forceinline__ VScale v_scale(float vs) {
    const bool none = vs < 1.17549435e-38f;
    vs = none ? 8.673617379884035e-19f : vs;
    return VScale{__builtin_amdgcn_logf(vs), __builtin_amdgcn_rcpf(vs), none};
}
// The denominator's unit. sum p' / vs is the softmax's sum in units of 2^M, but M follows
// s + log2 vs: beside small scales the sum would leave fp32's range (keys of scale 2^-120
// alone: 2^127 each). It is held in units of 2^(M - en), en a whole number per row: 0, or
// M - n where M lies more than 2^64 below n, the largest score (log2, or the sum's own
// log2); kept as g = 2^en, by which 1 / vs is multiplied. g is formed again for each tile
// with a scale below 2^-85 or while a g of the wave is not 1: else a term stays below 2^100,
// as p' does below 2^15. (Large scales need none: 2^-120 of a unit still has its 24 bits.)
constexpr float kUnitSlack = 64.f, kInvTop = 3.8685626e25f;  // 2^85
__device__ __forceinline__ float sum_unit(float d) {  // of d = M - n
    const float e = d < -kUnitSlack && d > -1e30f ? fmaxf(__builtin_rintf(d), -120.f) : 0.f;
    return __builtin_amdgcn_ldexpf(1.f, int(e));
}
__device__ __forceinline__ int unit_exp(float g) { return int(__float_as_uint(g) >> 23) - 127; }
__device__ __forceinline__ unsigned pack_f16(float lo, float hi) {
    f16x2 v;
    v[0] = (_Float16)lo;  // nearest, ties to even
    v[1] = (_Float16)hi;
    return __builtin_bit_cast(unsigned, v);
}
// Two probabilities as word w of the NV parts of a B operand (one: fp16; three: bf16), and
// 16 of them as the operands of the two products with V's 16 tokens.
template <int NV>
__device__ __forceinline__ void pack_pair(float lo, float hi, u32x4 (&f)[NV], int w) {
    if constexpr (NV == 1) {
        f[0][w] = pack_f16(lo, hi);
    } else {
        unsigned u[3];
        split3(lo, hi, u);
#pragma unroll
        for (int k = 0; k < 3; ++k) f[k][w] = u[k];
    }
}
template <int NV>
__device__ __forceinline__ void pack_p(const float* p, u32x4 (*f)[NV]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) pack_pair<NV>(p[2 * j], p[2 * j + 1], f[j / 4], j % 4);
}

template <bool FP8>
__device__ __forceinline__ u32x4 to_f16(unsigned a, unsigned b) {
    const u32x2 x = Code<FP8>::dec4_f16(a), y = Code<FP8>::dec4_f16(b);
    return u32x4{x[0], x[1], y[0], y[1]};
}
template <bool FP8>
__device__ __forceinline__ u32x4 to_bf16(unsigned a, unsigned b) {
    const u32x2 x = Code<FP8>::dec4_bf16(a), y = Code<FP8>::dec4_bf16(b);
    return u32x4{x[0], x[1], y[0], y[1]};
}
// V's codes as the probabilities' parts need them, and the product with one part
template <bool FP8, int NV>
__device__ __forceinline__ u32x4 v_operand(unsigned a, unsigned b) {
    if constexpr (NV == 1) return to_f16<FP8>(a, b);
    else return to_bf16<FP8>(a, b);
}
template <int NV>
__device__ __forceinline__ floatx4 mfma_v(u32x4 v, u32x4 p, floatx4 c) {
    if constexpr (NV == 1) return mfma_f16(v, p, c);
    else return mfma(v, p, c);
}

// The larger of a lane's value and of the lanes 16 and 32 away (the four lanes
// that share lane % 16), and their sum: register row swaps, no LDS round trip.
__device__ __forceinline__ float quad_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

}  // namespace
}  // namespace m3
