// m3_kv_attend_parts.hip -- attention of few rows a sequence behind prefixes that sequences share.
//
// A softmax over keys in two parts is joined from their sums: with (m, l, o) the unit, the
// probabilities' sum and the weighted values of each, o = (sum 2^(m - M) o) / (sum 2^(m - M) l).
// So a group's prefix is one more run of keys, whose rows are all its sequences' rows: read once
// for as many of them as a row tile holds, where every sequence would read it for a few rows.
// While that is little work, the groups' row tiles and the sequences' are items of one launch of
// the kernel for few rows, dealt out in even shares, and a merge takes a row's parts of both in
// their order. Above, the prefix goes through the kernel for many rows first; then workgroups
// that hold a sequence's own keys whole join its rows themselves, or again the merge does. (The plan's
// rules stand with it, m3_attn_host.cpp.)
//
// 16 heads over 4 of 128: 16 steps behind 8192 tokens (int8) 18 us and the merge's 5.7, where latencies
// decide: 3.4 us until the shares are known, 10 until a first tile is through, 1.6 a tile. 128 steps
// behind 8192 tokens, 63 .. 1023 of their own (e4m3): prefix 31 us, own keys and the joining 22, of them
// 14 the own keys' bytes; each sequence by itself 129. The prefix's parts are in fp32, 17 MB of them here.
#include "m3_attend_rows.h"

namespace m3 {
namespace {

// Parts p = 0 .. n - 1 of a row: the first at p0, the others at p1 + p * step.
struct Run {
    int n;
    int64_t p0, p1, step;
    __device__ __forceinline__ int64_t at(int p) const { return p ? p1 + p * step : p0; }
};
// Of an item of even shares, for key head h (of `heads`); solo: where it lies if one share holds it.
__device__ __forceinline__ Run run_of(const AttendDev& a, int e, int h, int rin, int64_t solo) {
    const int share = a.shares[0], f = a.shares[1 + e], n = a.shares[2 + e] - f;
    if (n <= 0) return Run{0, 0, 0, 0};
    const int64_t x0 = int64_t(a.c.heads) * f + int64_t(h) * n;
    const int64_t w0 = x0 / share, w1 = (x0 + n - 1) / share;
    if (w0 == w1) return Run{1, solo, 0, 0};
    return Run{int(w1 - w0) + 1, a.slots + (2 * w0 + 1) * a.rows + rin, a.slots + 2 * w0 * a.rows + rin, 2 * int64_t(a.rows)};
}

template <typename T>
__global__ __launch_bounds__(256) void attend_merge_kernel(AttendDev a, int team) {
    __shared__ __align__(16) float o_lds[256 * 4];
    const int D = a.D, width = D <= 128 ? 32 : 64, crews = 256 / width;
    const int crew = threadIdx.x / width, lane = threadIdx.x % width, member = crew % team;
    const int64_t at = int64_t(block_id()) * (crews / team) + crew / team;
    bool live = at < a.b.tokens * a.q_heads;
    const int64_t tok = live ? at / a.q_heads : 0;
    const int head = live ? int(at - tok * a.q_heads) : 0, h = head / a.group;
    int64_t i = tok;
    if (a.b.cu_q) {  // the last sequence that begins at or before the row
        int64_t lo = 0, hi = a.b.batch - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (a.b.cu_q[mid] <= tok) lo = mid;
            else hi = mid - 1;
        }
        i = lo;
    }
    const Seq sq = seq_of(a.b, i);
    const int64_t t = tok - sq.row0;
    live = live && t >= 0 && t < sq.n;
    Run pre{0, 0, 0, 0}, own{0, 0, 0, 0};
    if (live) {
        const int64_t g = group_of(a, i);
        if (g >= 0) {
            const Group gr = group_at(a, g);
            const int64_t r = (tok - gr.row0) * a.group + head % a.group;
            if (tok >= gr.row0 && tok - gr.row0 < gr.n) {
                if (a.splits_a) {
                    const int n = (gr.held + kTile - 1) / kTile;
                    pre = Run{n ? cut_of(n, a.splits_a, kPrefixPiece).pieces : 0, at, at, a.b.tokens * a.q_heads};
                } else {
                    pre = run_of(a, int(group_pair_at(a, g, r / a.rows)), h, int(r % a.rows), a.solo_a + at);
                }
            }
        }
        const int r = int(t) * a.group + head % a.group;
        own = run_of(a, a.items_a + int(pair_at(a, i, r / a.rows)), h, r % a.rows, a.solo_b + at);
    }
    const int parts = pre.n + own.n;
    auto place = [&](int p) { return p < pre.n ? pre.at(p) : own.at(p - pre.n); };
    // the first two parts of this crew are on their way while the units' maximum is found
    const float* po = a.part_o + 4 * lane;
    const bool mine = 4 * lane < D;
    floatx4 early[2];
    float unit[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int p = member + k * team;
        early[k] = floatx4{0, 0, 0, 0};
        unit[k] = -INFINITY;
        if (p < parts) {
            unit[k] = a.part_ml[2 * place(p)];
            if (mine) early[k] = *reinterpret_cast<const floatx4*>(po + place(p) * D);
        }
    }
    float2 own_ml{-INFINITY, 0.f};
    if (lane < parts) own_ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * place(lane));
    float m = own_ml.x;
    for (int p = lane + width; p < parts; p += width) m = fmaxf(m, a.part_ml[2 * place(p)]);
    for (int x = 1; x < width; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    float l = own_ml.x == -INFINITY ? own_ml.y : own_ml.y * __builtin_amdgcn_exp2f(own_ml.x - m);
    for (int p = lane + width; p < parts; p += width) {
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * place(p));
        l += ml.x == -INFINITY ? ml.y : ml.y * __builtin_amdgcn_exp2f(ml.x - m);
    }
    for (int x = 1; x < width; x <<= 1) l += __shfl_xor(l, x);
    floatx4 v{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) v += early[k] * (unit[k] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(unit[k] - m));
    if (mine) {
#pragma unroll 4
        for (int p = member + 2 * team; p < parts; p += team) {
            const float mp = a.part_ml[2 * place(p)];
            const float f = mp == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mp - m);
            v += *reinterpret_cast<const floatx4*>(po + place(p) * D) * f;
        }
    }
    if (team > 1) {
        *reinterpret_cast<floatx4*>(&o_lds[threadIdx.x * 4]) = v;
        __syncthreads();
        if (member == 0)
            for (int k = 1; k < team; ++k) v += *reinterpret_cast<const floatx4*>(&o_lds[(threadIdx.x + k * width) * 4]);
    }
    if (!live || member) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (4 * lane < D) {
        T* out = static_cast<T*>(a.out) + at * D + 4 * lane;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<u32x2*>(out) = u32x2{pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv)};
        else
            *reinterpret_cast<floatx4*>(out) = v * inv;
    }
    if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : m * kLn2 + __logf(l);
}

}  // namespace

hipError_t launch_rows_parts(const AttendDev& d, m3_dtype io, hipStream_t s) { return launch_rows_form<kParts>(d, io, s); }

hipError_t launch_merge(const AttendDev& d, m3_dtype io, hipStream_t s) {
    const JoinGrid g = join_grid(d);
    if (io == M3_BF16) hipLaunchKernelGGL((attend_merge_kernel<bf16_t>), g.grid, dim3(256), 0, s, d, g.team);
    else hipLaunchKernelGGL((attend_merge_kernel<float>), g.grid, dim3(256), 0, s, d, g.team);
    return hipGetLastError();
}

}  // namespace m3
