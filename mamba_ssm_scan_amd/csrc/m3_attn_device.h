// m3_attn_device.h -- device helpers shared by the attention layer's kernels:
// angles, 8-bit codes, rows of a ragged batch, cache addresses.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/m3_attn.h"
#include "m3_device.h"

namespace m3 {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
    bf16x2 v;
    v[0] = (__bf16)lo;  // nearest, ties to even
    v[1] = (__bf16)hi;
    return __builtin_bit_cast(unsigned, v);
}

// (m cos theta, m sin theta) of theta = pos * f, rounded to fp32 once. All in
// fp64, at half the fp32 rate here and needed once per (token, pair), not per
// head: pos * f has 55 bits, so an fp32 angle would lose whole turns at late
// positions. theta = k pi/2 + r with pi/2 in two doubles (the first step exact
// by fma, k < 2^31), then the Taylor series on |r| <= pi/4, whose first omitted
// terms are below 1e-19.
__device__ __forceinline__ void cos_sin(int32_t pos, float f, double m, float* c, float* s) {
    const double th = double(pos) * double(f);
    const double k = __builtin_rint(th * 0.63661977236758134308);
    double r = __builtin_fma(-k, 1.57079632679489655800, th);
    r = __builtin_fma(-k, 6.12323399573676603587e-17, r);
    const double z = r * r;
    double a = 1.0 / 355687428096000.0;               // 1 / 17!
    a = __builtin_fma(a, z, -1.0 / 1307674368000.0);  // 15!
    a = __builtin_fma(a, z, 1.0 / 6227020800.0);
    a = __builtin_fma(a, z, -1.0 / 39916800.0);
    a = __builtin_fma(a, z, 1.0 / 362880.0);
    a = __builtin_fma(a, z, -1.0 / 5040.0);
    a = __builtin_fma(a, z, 1.0 / 120.0);
    a = __builtin_fma(a, z, -1.0 / 6.0);
    const double sr = __builtin_fma(a * z, r, r);
    double b = -1.0 / 6402373705728000.0;             // 1 / 18!
    b = __builtin_fma(b, z, 1.0 / 20922789888000.0);  // 16!
    b = __builtin_fma(b, z, -1.0 / 87178291200.0);
    b = __builtin_fma(b, z, 1.0 / 479001600.0);
    b = __builtin_fma(b, z, -1.0 / 3628800.0);
    b = __builtin_fma(b, z, 1.0 / 40320.0);
    b = __builtin_fma(b, z, -1.0 / 720.0);
    b = __builtin_fma(b, z, 1.0 / 24.0);
    b = __builtin_fma(b, z, -0.5);
    const double cr = __builtin_fma(b, z, 1.0);
    const int q = int(int64_t(k) & 3);
    const double ss = (q & 1) ? cr : sr, cc = (q & 1) ? sr : cr;
    *s = float(m * ((q & 2) ? -ss : ss));
    *c = float(m * (((q + 1) & 2) ? -cc : cc));
}

// A launch of `blocks` workgroups (below 2^31): the first dimension holds fewer than 2^32
// threads, so what is beyond 2^22 workgroups goes on along the third. The last may be
// beyond `blocks`: every kernel returns where its index is.
inline dim3 grid_of(int64_t blocks, unsigned y = 1) {
    const int64_t x = int64_t(1) << 22;
    return blocks <= x ? dim3(unsigned(blocks), y) : dim3(unsigned(x), y, unsigned((blocks + x - 1) / x));
}
__device__ __forceinline__ unsigned block_id() { return (blockIdx.z << 22) + blockIdx.x; }

// One pair turned by (c, s). The products are rounded one by one (no fma): the
// result is then the same wherever a pair is turned, and the codes that the
// cache holds are those of the formula as written.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
#pragma clang fp contract(off)
    const float ac = a * c, bs = b * s, as = a * s, bc = b * c;
    a = ac - bs;
    b = as + bc;
}

// 8 entries of a row. Wide: one or two 16-byte accesses; else entry by entry.
template <bool WIDE>
__device__ __forceinline__ void load8(const bf16_t* p, float* v) {
    if constexpr (WIDE) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = bf16_to_f32(p[j].bits);
    }
}
template <bool WIDE>
__device__ __forceinline__ void load8(const float* p, float* v) {
    if constexpr (WIDE) {
        const floatx4 a = *reinterpret_cast<const floatx4*>(p), b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p[j];
    }
}
template <bool WIDE>
__device__ __forceinline__ void store8(bf16_t* p, const float* v) {
    if constexpr (WIDE) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<u32x4*>(p) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j].bits = f32_to_bf16(v[j]);
    }
}
template <bool WIDE>
__device__ __forceinline__ void store8(float* p, const float* v) {
    if constexpr (WIDE) {
        *reinterpret_cast<floatx4*>(p) = floatx4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4*>(p + 4) = floatx4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = v[j];
    }
}

// 8-bit codes. enc4: four values already divided by the scale, held to the
// format's range, to the nearest code (ties to even). dec4: four codes as fp32;
// dec4_bf16, dec4_f16: as packed bf16 or fp16 (both formats are exact in both).
template <bool FP8>
struct Code;
template <>
struct Code<true> {
    static constexpr float kTop = 448.f;
    __device__ __forceinline__ static unsigned enc4(float a, float b, float c, float d) {
        a = __builtin_amdgcn_fmed3f(a, -kTop, kTop);
        b = __builtin_amdgcn_fmed3f(b, -kTop, kTop);
        c = __builtin_amdgcn_fmed3f(c, -kTop, kTop);
        d = __builtin_amdgcn_fmed3f(d, -kTop, kTop);
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return unsigned(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
    }
    __device__ __forceinline__ static void dec4(unsigned w, float* v) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
        v[0] = lo[0];
        v[1] = lo[1];
        v[2] = hi[0];
        v[3] = hi[1];
    }
    __device__ __forceinline__ static u32x2 dec4_bf16(unsigned w) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
        return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
    }
    __device__ __forceinline__ static u32x2 dec4_f16(unsigned w) {
        const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false);
        const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true);
        return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
    }
};
template <>
struct Code<false> {
    static constexpr float kTop = 127.f;
    __device__ __forceinline__ static unsigned one(float a) {
        return unsigned(int(__builtin_rintf(__builtin_amdgcn_fmed3f(a, -kTop, kTop)))) & 0xffu;
    }
    __device__ __forceinline__ static unsigned enc4(float a, float b, float c, float d) {
        return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
    }
    __device__ __forceinline__ static void dec4(unsigned w, float* v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = float(int8_t(w >> (8 * j)));
    }
    __device__ __forceinline__ static u32x2 dec4_bf16(unsigned w) {
        float v[4];
        dec4(w, v);
        return u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
    // code + 128 = u as the low byte of the fp16 number 1024 + u, less 1152
    __device__ __forceinline__ static u32x2 dec4_f16(unsigned w) {
        const unsigned u = w ^ 0x80808080u;
        const f16x2 off{_Float16(-1152.f), _Float16(-1152.f)};
        const f16x2 lo = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + off;
        const f16x2 hi = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + off;
        return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
    }
};

// Rows of a sequence of the batch, held inside [0, tokens) whatever the device arrays
// hold. Rows beyond max_q are left out; those before them keep their positions.
struct Seq {
    int64_t row0;  // its first row
    int n;         // its rows, max_q at most
    int held;      // tokens held once all its rows are in (>= 0)
    int base;      // position of its first row (negative: more rows than tokens held)
};
__device__ __forceinline__ Seq seq_of(const m3_kv_batch& b, int64_t i) {
    Seq s;
    s.held = max(b.kv_len[i], 0);
    if (b.cu_q) {
        const int64_t lo = min(max(int64_t(b.cu_q[i]), int64_t(0)), b.tokens);
        const int64_t hi = min(max(int64_t(b.cu_q[i + 1]), lo), b.tokens);
        s.row0 = lo;
        s.n = int(min(hi - lo, b.max_q));
        s.base = s.held - int(hi - lo);
    } else {
        s.row0 = i;
        s.n = 1;
        s.base = s.held - 1;
    }
    return s;
}

// Units of a ragged batch -- tiles of 2^shift (row, head of a group) pairs, or blocks of
// tokens -- one after the other. Sequence i's begin at (cu_q[i] per >> shift) + extra i, which
// leaves it the units of its rows (and of a first one begun before them, with extra 2), and
// ends are found by a search of cu_q: a launch has work for nearly all its workgroups
// however loose max_q is. `at`: the unit among its sequence's (negative or beyond its
// rows: none; cu_q may be anything).
__device__ __forceinline__ int64_t first_unit(const m3_kv_batch& b, int64_t i, int per, int shift, int extra) {
    return (min(max(int64_t(b.cu_q[i]), int64_t(0)), b.tokens) * per >> shift) + extra * i;
}
struct Unit {
    int64_t i, at;
};
__device__ __forceinline__ Unit unit_of(const m3_kv_batch& b, int64_t e, int per, int shift, int extra) {
    int64_t lo = 0, hi = b.batch - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (first_unit(b, mid, per, shift, extra) <= e) lo = mid;
        else hi = mid - 1;
    }
    return Unit{lo, e - first_unit(b, lo, per, shift, extra)};
}

// Where block `blk` (16 tokens) of a sequence is held: its index among all
// (page, head 0) blocks, or -1 where no page holds it. shift: log2(page_size / 16).
__device__ __forceinline__ int64_t block_at(const int32_t* pages, int64_t max_pages, int64_t num_pages, int shift,
                                            int heads, int64_t blk) {
    const int64_t pi = blk >> shift;
    if (blk < 0 || pi >= max_pages) return -1;
    const int64_t p = pages[pi];
    if (p < 0 || p >= num_pages) return -1;
    return ((p * heads) << shift) + (blk & ((int64_t(1) << shift) - 1));
}

}  // namespace
}  // namespace m3
