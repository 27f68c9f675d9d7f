// m3_kv_append.hip -- new keys and values into the paged 8-bit cache, the keys
// (and the queries) turned on the way; and the cache's values read back.
//
// Per touched block of 16 tokens and head: s' = max(old ? s : 0, max|new| / Q),
// code = nearest(x / s'). Memory-bound: the new rows are read once and their
// codes written once, old codes are read only in the block a sequence was in the
// middle of. A workgroup takes one block of one sequence; the (cos, sin) of its
// tokens are formed once (fp64) and shared by its jobs: K and V of each cache
// head and the query heads, one job a wave at a time, dealt over blockIdx.y when
// the blocks alone would leave the chip idle (single tokens).
//
// The maximum has to be known before the first code, so a job holds its rows: wide
// rows in registers, each lane pieces of 8 entries with their partners in the
// rotation; V then crosses LDS once, as its codes lie transposed ([entry][token], so
// that attention reads 16 tokens of an entry with one load). Other rows go through the
// wave's own LDS rows in fp32. Waves never wait for each other after the angles.
//
// 4 prompts of 2048 (4 heads of 128 and 16 query heads, e4m3): 24 us, 3.8 TB/s of reads
// and writes (31 us where half of each head turns in the half layout: too many registers as
// pairs, so keys and queries go through LDS); one token of each of 128 sequences: 5.6 us.
// Reading a cache back: 9.1 us for the values of those prompts (25 MB), 7.8 us for the
// last block of 128 sequences.
#include <algorithm>

#include "m3_attn_device.h"
#include "m3_attn_internal.h"

namespace m3 {
namespace {

struct AppendDev {
    m3_kv_cache c;
    m3_kv_batch b;
    m3_rows k, v, q, qo;
    int q_heads, D, half, interleaved, shift, nblk, k_slices, v_slices;  // nblk 0: blocks one after the other (unit_of)
    int kq_jobs, v_jobs;      // register jobs of a row (0: the rows go through LDS)
    unsigned kq_inv, v_inv;   // ceil(2^16 / jobs): e / jobs = e * inv >> 16 for e < 512
    float mscale;
    const float* inv_freq;
};

__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
__device__ __forceinline__ unsigned wave_umax(unsigned v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = max(v, unsigned(__shfl_xor(int(v), m)));
    return v;
}
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Rows lo .. hi - 1 of a job into LDS (fp32), turned where cs is given; returns
// the lane's largest magnitude as bits (above any finite one for inf and NaN).
template <typename T, bool WIDE>
__device__ __forceinline__ unsigned gather(const AppendDev& a, const T* src, int64_t tok, int lo, int hi, float* rows,
                                           const float2* cs, int lane) {
    const int D = a.D, per = D / 8;
    const int rot = cs ? 2 * a.half : 0;
    unsigned top = 0;
    for (int e = lane; e < (hi - lo) * per; e += 64) {
        const int s = e / per, d = 8 * (e - s * per);
        float v[8];
        load8<WIDE>(src + s * tok + d, v);
        float* o = rows + (lo + s) * D + d;
        *reinterpret_cast<floatx4*>(o) = floatx4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4*>(o + 4) = floatx4{v[4], v[5], v[6], v[7]};
#pragma unroll
        for (int j = 0; j < 8; ++j) top = d + j >= rot ? max(top, mag(v[j])) : top;
    }
    wave_fence();
    if (rot) {
        for (int e = lane; e < (hi - lo) * a.half; e += 64) {
            const int s = e / a.half, i = e - s * a.half;
            const int i0 = a.interleaved ? 2 * i : i, i1 = a.interleaved ? 2 * i + 1 : i + a.half;
            float* o = rows + (lo + s) * D;
            float u = o[i0], v = o[i1];
            const float2 w = cs[(lo + s) * a.half + i];
            turn(u, v, w.x, w.y);
            o[i0] = u;
            o[i1] = v;
            top = max(top, max(mag(u), mag(v)));
        }
        wave_fence();
    }
    return top;
}

// A job's rows in registers. Job e of the (hi - lo) * jobs of the rows is piece
// e % jobs (8 entries) of row e / jobs, or, with pairs (half layout), that piece and
// its partner half further on; pieces after rot stand alone. A lane holds jobs lane,
// lane + 64, ...; loads beyond the last job repeat it, so that none is behind a branch.
// N: entries a lane holds, 32 for headdim up to 128, else 64.
template <bool PAIRS, int N>
struct Held {
    static constexpr int kEach = PAIRS ? 16 : 8, kN = N / kEach;
    float v[kN][kEach];
};
struct Job {
    int s, d, two;  // row, first entry, whether the partner belongs to it
};
template <bool PAIRS>
__device__ __forceinline__ Job job_of(const AppendDev& a, int e, int jobs, unsigned inv) {
    const int s = int(unsigned(e) * inv >> 16), j = e - s * jobs;
    if constexpr (PAIRS) {
        const int turned = a.half / 8;
        return Job{s, j < turned ? 8 * j : 8 * (j + turned), j < turned};
    } else {
        return Job{s, 8 * j, 0};
    }
}
template <typename T, bool PAIRS, int N>
__device__ __forceinline__ void fetch(const AppendDev& a, const T* src, int64_t tok, int n, int jobs, unsigned inv,
                                      int lane, Held<PAIRS, N>& r) {
#pragma unroll
    for (int k = 0; k < (Held<PAIRS, N>::kN); ++k) {
        if (64 * k >= n * jobs) break;  // (the wave as a whole)
        const Job b = job_of<PAIRS>(a, min(lane + 64 * k, n * jobs - 1), jobs, inv);
        const T* p = src + b.s * tok + b.d;
        load8<true>(p, r.v[k]);
        if constexpr (PAIRS) load8<true>(p + (b.two ? a.half : 0), r.v[k] + 8);
    }
}
// turned by cs (rows lo ..), and the largest magnitude's bits
template <bool PAIRS, int N>
__device__ __forceinline__ unsigned turn_held(const AppendDev& a, const float2* cs, int n, int jobs, unsigned inv,
                                              int lane, Held<PAIRS, N>& r) {
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < (Held<PAIRS, N>::kN); ++k) {
        if (64 * k >= n * jobs) break;
        const Job b = job_of<PAIRS>(a, min(lane + 64 * k, n * jobs - 1), jobs, inv);
        float* v = r.v[k];
        if constexpr (PAIRS) {
            if (cs && b.two) {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float2 w = cs[b.s * a.half + b.d + x];
                    turn(v[x], v[8 + x], w.x, w.y);
                }
            }
#pragma unroll
            for (int x = 8; x < 16; ++x) top = max(top, mag(v[x]));  // (alone: the piece twice)
        } else if (cs && b.d < 2 * a.half) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 w = cs[b.s * a.half + b.d / 2 + x];
                turn(v[2 * x], v[2 * x + 1], w.x, w.y);
            }
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) top = max(top, mag(v[x]));
        __builtin_amdgcn_sched_barrier(0);  // (one job's angles at a time)
    }
    return top;
}
// What a job does with each piece it holds: at(row, first entry, 8 values).
template <bool PAIRS, int N, typename F>
__device__ __forceinline__ void each_piece(const AppendDev& a, int n, int jobs, unsigned inv, int lane, Held<PAIRS, N>& r,
                                           F at) {
#pragma unroll
    for (int k = 0; k < (Held<PAIRS, N>::kN); ++k) {
        const int e = lane + 64 * k;
        if (e >= n * jobs) continue;
        const Job b = job_of<PAIRS>(a, e, jobs, inv);
        at(b.s, b.d, r.v[k]);
        if constexpr (PAIRS)
            if (b.two) at(b.s, b.d + a.half, r.v[k] + 8);
    }
}

// The scale of a block from its old one and the largest new magnitude.
struct Scale {
    float s, inv;  // stored scale; 1 / s, or 0 where nothing can be held (s 0 or not finite)
};
template <bool FP8>
__device__ __forceinline__ Scale new_scale(float old, unsigned top) {
    const unsigned m = max(mag(old), mag(__uint_as_float(top) * (1.f / Code<FP8>::kTop)));
    Scale r{__uint_as_float(m), 0.f};
    if (m >= 0x7f800000u)
        r.s = __uint_as_float(0x7fc00000u);
    else if (m < 0x00800000u)  // below the normal numbers: 1 / s could overflow
        r.s = 0.f;
    else
        r.inv = 1.f / r.s;
    return r;
}

// 16 codes from 16 fp32 values at p, stride st, times f
template <bool FP8>
__device__ __forceinline__ u32x4 codes16(const float* p, int st, float f) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = Code<FP8>::enc4(p[(4 * j) * st] * f, p[(4 * j + 1) * st] * f, p[(4 * j + 2) * st] * f,
                               p[(4 * j + 3) * st] * f);
    return w;
}
template <bool FP8>
__device__ __forceinline__ u32x4 recode16(u32x4 w, float ratio) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[4];
        Code<FP8>::dec4(w[j], v);
        w[j] = Code<FP8>::enc4(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
    }
    return w;
}

// A workgroup's block: slots lo .. hi - 1 of it are new, row the batch's row of the
// first, at its index in the cache (head 0; -1: no page), begun: it holds older tokens.
struct Where {
    int lo, hi;
    int64_t row, at;
    bool begun;
};

template <typename T, bool WIDE, int REG, int N>
__device__ __forceinline__ void put_query(const AppendDev& a, const Where& w, int h, const float2* cs, float* rows,
                                          int lane) {
    const T* src = static_cast<const T*>(a.q.p) + w.row * a.q.token_stride + h * a.q.head_stride;
    T* dst = static_cast<T*>(a.qo.p) + w.row * a.qo.token_stride + h * a.qo.head_stride;
    const int n = w.hi - w.lo, D = a.D;
    if constexpr (REG > 0) {
        Held<REG == 2, N> r;
        fetch<T>(a, src, a.q.token_stride, n, a.kq_jobs, a.kq_inv, lane, r);
        turn_held(a, cs ? cs + w.lo * a.half : nullptr, n, a.kq_jobs, a.kq_inv, lane, r);
        each_piece(a, n, a.kq_jobs, a.kq_inv, lane, r,
                   [&](int s, int d, const float* v) { store8<true>(dst + s * a.qo.token_stride + d, v); });
    } else {
        gather<T, WIDE>(a, src, a.q.token_stride, w.lo, w.hi, rows, cs, lane);
        for (int e = lane; e < n * (D / 8); e += 64) {
            const int s = e / (D / 8), d = 8 * (e - s * (D / 8));
            store8<WIDE>(dst + s * a.qo.token_stride + d, rows + (w.lo + s) * D + d);
        }
        wave_fence();
    }
}

template <typename T, bool FP8, bool WIDE, int REG, int N>
__device__ __forceinline__ void put_key(const AppendDev& a, const Where& w, int h, const float2* cs, float* rows,
                                        int lane) {
    const int64_t slot = w.at + (int64_t(h) << a.shift);
    const int lo = w.lo, hi = w.hi, n = hi - lo, D = a.D, per = D / 16;
    char* code = static_cast<char*>(a.c.k) + slot * 16 * D;
    const T* src = static_cast<const T*>(a.k.p) + w.row * a.k.token_stride + h * a.k.head_stride;
    const float old = w.begun ? a.c.k_scale[slot] : 0.f;
    unsigned top;
    Held<REG == 2, N> r;
    if constexpr (REG > 0) {
        fetch<T>(a, src, a.k.token_stride, n, a.kq_jobs, a.kq_inv, lane, r);
        top = turn_held(a, cs ? cs + lo * a.half : nullptr, n, a.kq_jobs, a.kq_inv, lane, r);
    } else {
        top = gather<T, WIDE>(a, src, a.k.token_stride, lo, hi, rows, cs, lane);
    }
    const Scale ns = new_scale<FP8>(old, wave_umax(top));
    const bool none = ns.inv == 0.f, all = !w.begun || __float_as_uint(ns.s) != __float_as_uint(old);
    if constexpr (REG > 0) {
        each_piece(a, n, a.kq_jobs, a.kq_inv, lane, r, [&](int s, int d, const float* v) {
            const float i = ns.inv;
            u32x2 c{Code<FP8>::enc4(v[0] * i, v[1] * i, v[2] * i, v[3] * i),
                    Code<FP8>::enc4(v[4] * i, v[5] * i, v[6] * i, v[7] * i)};
            if (none) c = u32x2{0, 0};
            *reinterpret_cast<u32x2*>(code + (lo + s) * D + d) = c;
        });
    } else {
        for (int e = lane; e < n * per; e += 64) {
            const int s = lo + e / per, d = 16 * (e % per);
            *reinterpret_cast<u32x4*>(code + s * D + d) =
                none ? u32x4{0, 0, 0, 0} : codes16<FP8>(rows + s * D + d, 1, ns.inv);
        }
    }
    if (all) {  // the other slots too: older codes where the scale grew, 0 after the end
        const float ratio = none ? 0.f : old * ns.inv;
        for (int e = lane; e < (16 - n) * per; e += 64) {
            const int f = e / per, s = f < lo ? f : f + n;
            u32x4* c = reinterpret_cast<u32x4*>(code + s * D + 16 * (e % per));
            *c = s < lo && !none ? recode16<FP8>(*c, ratio) : u32x4{0, 0, 0, 0};
        }
    }
    if (lane == 0) a.c.k_scale[slot] = ns.s;
    wave_fence();
}

template <typename T, bool FP8, bool WIDE, int REG, int N>
__device__ __forceinline__ void put_value(const AppendDev& a, const Where& w, int h, float* rows, int lane) {
    const int64_t slot = w.at + (int64_t(h) << a.shift);
    const int lo = w.lo, hi = w.hi, n = hi - lo, D = a.D;
    u32x4* code = reinterpret_cast<u32x4*>(static_cast<char*>(a.c.v) + slot * 16 * D);
    const T* src = static_cast<const T*>(a.v.p) + w.row * a.v.token_stride + h * a.v.head_stride;
    const float old = w.begun ? a.c.v_scale[slot] : 0.f;
    unsigned top;
    if constexpr (REG > 0) {
        Held<false, N> r;
        fetch<T>(a, src, a.v.token_stride, n, a.v_jobs, a.v_inv, lane, r);
        top = turn_held(a, static_cast<const float2*>(nullptr), n, a.v_jobs, a.v_inv, lane, r);
        each_piece(a, n, a.v_jobs, a.v_inv, lane, r,
                   [&](int s, int d, const float* v) { store8<true>(rows + (lo + s) * D + d, v); });
        wave_fence();
    } else {
        top = gather<T, WIDE>(a, src, a.v.token_stride, lo, hi, rows, nullptr, lane);
    }
    const Scale ns = new_scale<FP8>(old, wave_umax(top));
    const bool none = ns.inv == 0.f, grown = __float_as_uint(ns.s) != __float_as_uint(old);
    const float ratio = none ? 0.f : old * ns.inv;
    // 16 slots of one entry a lane; old slots keep their byte unless the scale grew
    for (int d = lane; d < D; d += 64) {
        u32x4 c = w.begun ? code[d] : u32x4{0, 0, 0, 0};
        if (w.begun && grown) c = none ? u32x4{0, 0, 0, 0} : recode16<FP8>(c, ratio);
        const u32x4 f = none ? u32x4{0, 0, 0, 0} : codes16<FP8>(rows + d, D, ns.inv);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int l = min(max(lo - 4 * b, 0), 4), u = min(max(hi - 4 * b, 0), 4);
            const unsigned below = l == 4 ? ~0u : (1u << (8 * l)) - 1u;
            const unsigned upto = u == 4 ? ~0u : (1u << (8 * u)) - 1u;
            c[b] = (c[b] & below) | (f[b] & upto & ~below);
        }
        code[d] = c;
    }
    if (lane == 0) a.c.v_scale[slot] = ns.s;
    wave_fence();
}

// REG: 0 the rows go through LDS (any rotation, stride and alignment); 1, 2 wide rows
// held in registers, single pieces or pairs. blockIdx.y: slices of the key heads, then
// of the value heads, then of the query heads (a loop of its own each, or their
// invariants would all be held at once).
template <typename T, bool FP8, bool WIDE, int REG, int N>
__global__ __launch_bounds__(256, REG ? (N == 32 ? 4 : 2) : 1) void append_kernel(AppendDev a) {
    extern __shared__ __align__(16) float lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const unsigned id = block_id();
    const Unit u = a.nblk ? Unit{id / unsigned(a.nblk), id % unsigned(a.nblk)} : unit_of(a.b, id, 1, 4, 2);
    const int64_t i = u.i;
    if (i >= a.b.batch || u.at < 0) return;
    const Seq q = seq_of(a.b, i);
    const int64_t before = q.base;  // position of the sequence's first row (negative: not stored)
    const int64_t blk = (before >> 4) + u.at;
    Where w;
    w.lo = int(max(before - 16 * blk, int64_t(0)));
    w.hi = int(min(before + q.n - 16 * blk, int64_t(16)));
    if (w.hi <= w.lo) return;  // (the workgroup as a whole)
    w.row = q.row0 + (16 * blk + w.lo - before);
    w.begun = w.lo > 0 && blk * 16 < before;
    w.at = block_at(a.b.pages + i * a.b.max_pages, a.b.max_pages, a.c.num_pages, a.shift, a.c.heads, blk);

    float* rows = lds + wave * 16 * a.D;
    const int y = blockIdx.y;
    if (y >= a.k_slices && y < a.k_slices + a.v_slices) {
        if (w.at >= 0)
            for (int h = (y - a.k_slices) * waves + wave; h < a.c.heads; h += a.v_slices * waves)
                put_value<T, FP8, WIDE, REG, N>(a, w, h, rows, lane);
        return;
    }
    float2* cs = nullptr;
    if (a.inv_freq) {
        cs = reinterpret_cast<float2*>(lds + waves * 16 * a.D);
        for (int e = threadIdx.x; e < (w.hi - w.lo) * a.half; e += blockDim.x) {
            const int s = e / a.half, p = e - s * a.half;
            float c, sn;
            cos_sin(int32_t(16 * blk + w.lo + s), a.inv_freq[p], double(a.mscale), &c, &sn);
            cs[(w.lo + s) * a.half + p] = float2{c, sn};
        }
        __syncthreads();
    }
    if (y < a.k_slices) {
        if (w.at >= 0)
            for (int h = y * waves + wave; h < a.c.heads; h += a.k_slices * waves)
                put_key<T, FP8, WIDE, REG, N>(a, w, h, cs, rows, lane);
    } else {
        const int first = a.k_slices + a.v_slices, q_slices = gridDim.y - first;
        for (int h = (y - first) * waves + wave; h < a.q_heads; h += q_slices * waves)
            put_query<T, WIDE, REG, N>(a, w, h, cs, rows, lane);
    }
}

template <typename T, bool FP8>
hipError_t launch_append(const AppendArgs& a) {
    const AppendPlan plan = append_plan(a.b);
    AppendDev d{a.c, a.b, a.k, a.v, a.q, a.q_out, a.q.p ? a.q_heads : 0, a.c.headdim, a.rot.rot / 2,
                a.rot.interleaved, __builtin_ctz(unsigned(a.c.page_size / 16)), int(plan.each),
                0, 0, 0, 0, 0, 0, a.rot.mscale, a.rot.inv_freq};
    const int D = a.c.headdim, rot = a.rot.inv_freq ? a.rot.rot : 0;
    const bool pairs = rot && !a.rot.interleaved;
    int reg = a.wide && rot % (pairs ? 16 : 8) == 0 ? (pairs ? 2 : 1) : 0;
    d.kq_jobs = pairs ? (D - rot / 2) / 8 : D / 8;
    if (reg == 2 && d.kq_jobs > (D <= 128 ? 8 : 16)) reg = 0;  // (a short rotated part of a wide head: too many registers as pairs)
    d.v_jobs = D / 8;
    d.kq_inv = (65536u + d.kq_jobs - 1) / d.kq_jobs;
    d.v_inv = (65536u + d.v_jobs - 1) / d.v_jobs;
    const int64_t blocks = plan.blocks;
    const int waves = a.c.headdim <= 128 ? 4 : 2;  // LDS rows and angles within 64 KiB
    // heads of a wave: 1, or as many as leave about 4 workgroups a CU, 8 of fp32 rows
    // (4 prompts of 2048, 16 + 4 heads of 128: bf16 24.0 us and 25.0 with 8, fp32 43.0 with 4 and 40.7)
    const int64_t wide = blocks * (2 * a.c.heads + d.q_heads);
    const int each = int(std::min<int64_t>(16, std::max<int64_t>(1, wide / (512 * int64_t(sizeof(T)) * waves))));
    auto slices = [&](int heads) { return (heads + waves * each - 1) / (waves * each); };
    d.k_slices = d.v_slices = slices(a.c.heads);
    const int y = 2 * d.k_slices + slices(d.q_heads);
    const size_t lds = size_t(waves) * 16 * a.c.headdim * 4 + (a.rot.inv_freq ? size_t(16) * d.half * 8 : 0);
    const dim3 grid = grid_of(blocks, unsigned(y)), block{unsigned(64 * waves)};
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, a.stream, d); };
    if (reg == 2)
        D <= 128 ? launch(append_kernel<T, FP8, true, 2, 32>) : launch(append_kernel<T, FP8, true, 2, 64>);
    else if (reg == 1)
        D <= 128 ? launch(append_kernel<T, FP8, true, 1, 32>) : launch(append_kernel<T, FP8, true, 1, 64>);
    else if (a.wide)
        launch(append_kernel<T, FP8, true, 0, 32>);
    else
        launch(append_kernel<T, FP8, false, 0, 32>);
    return hipGetLastError();
}

struct ReadDev {
    m3_kv_cache c;
    const int32_t* first;
    const int32_t* count;
    const int32_t* pages;
    void* k_out;
    void* v_out;
    int64_t batch, max_pages, max_count;
    int D, shift, nblk;
};

// One block of positions of one sequence a workgroup, K or V of a head a wave.
// K: 16 entries of a row a lane. V: two entries' 16 tokens a lane, stored as
// pairs, so that a wave's store is whole lines of a row.
template <typename T, bool FP8>
__global__ __launch_bounds__(256) void read_kernel(ReadDev a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned id = block_id();
    const int64_t i = id / unsigned(a.nblk);
    if (i >= a.batch) return;
    const int64_t first = a.first[i], count = min(int64_t(max(a.count[i], 0)), a.max_count);
    const int64_t blk = (first >> 4) + id % unsigned(a.nblk);
    const int64_t j0 = 16 * blk - first;  // output row of slot 0
    const int H = a.c.heads, D = a.D;
    const int64_t at = block_at(a.pages + i * a.max_pages, a.max_pages, a.c.num_pages, a.shift, H, blk);
    for (int j = blockIdx.y * 4 + wave; j < 2 * H; j += gridDim.y * 4) {
        const bool is_v = j >= H;
        const int h = is_v ? j - H : j;
        const int64_t slot = at + (int64_t(h) << a.shift);
        T* out = static_cast<T*>(is_v ? a.v_out : a.k_out) + ((i * a.max_count + j0) * H + h) * int64_t(D);
        const char* code = static_cast<const char*>(is_v ? a.c.v : a.c.k) + slot * 16 * D;
        const bool any = at >= 0 && j0 < count && 16 * blk + 16 > 0;
        const float sc = any ? (is_v ? a.c.v_scale : a.c.k_scale)[slot] : 0.f;
        if (!is_v) {
            const int per = D / 16;
            for (int e = lane; e < 16 * per; e += 64) {
                const int s = e / per, d = 16 * (e - s * per);
                const int64_t r = j0 + s;
                if (r < 0 || r >= a.max_count) continue;
                float v[16];
                const bool live = any && r < count;
                const u32x4 w = live ? *reinterpret_cast<const u32x4*>(code + s * D + d) : u32x4{0, 0, 0, 0};
#pragma unroll
                for (int b = 0; b < 4; ++b) Code<FP8>::dec4(w[b], v + 4 * b);
#pragma unroll
                for (int b = 0; b < 16; ++b) v[b] = live ? v[b] * sc : 0.f;
                T* o = out + s * int64_t(H) * D + d;
                store8<true>(o, v);
                store8<true>(o + 8, v + 8);
            }
        } else {
            for (int d = 2 * lane; d < D; d += 128) {
                u32x4 w0{0, 0, 0, 0}, w1{0, 0, 0, 0};
                if (any) {
                    w0 = *reinterpret_cast<const u32x4*>(code + d * 16);
                    w1 = *reinterpret_cast<const u32x4*>(code + d * 16 + 16);
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float v0[4], v1[4];
                    Code<FP8>::dec4(w0[b], v0);
                    Code<FP8>::dec4(w1[b], v1);
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int64_t r = j0 + 4 * b + s;
                        if (r < 0 || r >= a.max_count) continue;
                        const bool live = any && r < count;
                        const float x = live ? v0[s] * sc : 0.f, y = live ? v1[s] * sc : 0.f;
                        T* o = out + (4 * b + s) * int64_t(H) * D + d;
                        if constexpr (sizeof(T) == 2)
                            *reinterpret_cast<unsigned*>(o) = pack_bf16(x, y);
                        else
                            *reinterpret_cast<float2*>(o) = float2{x, y};
                    }
                }
            }
        }
    }
}

template <typename T, bool FP8>
hipError_t launch_read(const ReadArgs& a) {
    ReadDev d{a.c, a.first, a.count, a.pages, a.k_out, a.v_out, a.batch, a.max_pages, a.max_count, a.c.headdim,
              __builtin_ctz(unsigned(a.c.page_size / 16)), int((a.max_count + 14) / 16 + 1)};
    const int64_t blocks = a.batch * d.nblk;
    const int slices = int(std::max<int64_t>(1, std::min<int64_t>((2 * a.c.heads + 3) / 4, 2048 / blocks)));
    const dim3 grid = grid_of(blocks, unsigned(slices));
    hipLaunchKernelGGL((read_kernel<T, FP8>), grid, dim3(256), 0, a.stream, d);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a) {
    const bool fp8 = a.c.format == M3_KV_FP8;
    if (a.io == M3_BF16) return fp8 ? launch_append<bf16_t, true>(a) : launch_append<bf16_t, false>(a);
    return fp8 ? launch_append<float, true>(a) : launch_append<float, false>(a);
}

hipError_t launch_kv_read(const ReadArgs& a) {
    const bool fp8 = a.c.format == M3_KV_FP8;
    if (a.io == M3_BF16) return fp8 ? launch_read<bf16_t, true>(a) : launch_read<bf16_t, false>(a);
    return fp8 ? launch_read<float, true>(a) : launch_read<float, false>(a);
}

}  // namespace m3
