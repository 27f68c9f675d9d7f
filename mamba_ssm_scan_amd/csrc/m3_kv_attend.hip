// m3_kv_attend.hip -- softmax attention over the paged 8-bit cache.
//
// o = sum_j p_j v_j with p the softmax of scale * q . k_j, in one pass over the
// keys with a running reference and sum (log2 domain): when the reference grows,
// what was summed is scaled down. The codes are exact in bf16 and fp16, so the
// products run on MFMA over the codes themselves, with the block scales applied in fp32:
// K's to the scores, V's as log2 vs in the probabilities' exponents. bf16 rows take q . k
// in bf16 and p . v in fp16 (p rounded to its 11 bits); fp32 rows and their probabilities
// are split into three bf16 parts each (24 bits), so that nothing is rounded to fewer.
//
// attend_rows_kernel. A workgroup takes up to 16 QT rows of one (sequence, key
// head) -- a row is a (token, head of the group) pair, so grouped heads share
// every key -- and one split of its keys; each of its 4 waves takes every fourth
// tile of 64 keys straight from memory into registers:
//   S^T = K Q^T   A = 16 keys, lane (r = l % 16, g = l / 16) loads a quarter of
//                 row r's codes; tile t's row r is key 16 (r / 4) + 4 t + r % 4,
//                 so the lane's 16 scores over the 4 tiles are those of the 16
//                 keys of block g, in order
//   O^T = V^T P^T the scores' registers are the B operand as they stand (no
//                 shuffle, no LDS), and the A operand is V's stored layout: 16
//                 tokens of an entry, one 16-byte load
// Each code is read from memory once per row tile, and the next tile's K and
// page numbers are requested before this tile's softmax.
//
// Bound by memory, one read of the keys and values seen: 4 sequences of 131072 tokens
// (4 heads of 128, e4m3) 102 us with the join, 5.3 TB/s; 128 sequences of 128 .. 4096
// tokens (int8) 70 us, 3.9 TB/s, where 128 of 2112 each reach 5.1: the longest of a
// workgroup's sequences decides. One sequence of 2048 is a chain of latencies (lengths,
// page, codes, then the join's launch, as its 32 tiles are split over workgroups of four
// waves): 8.4 and 4.4 us. 16 sequences of 8000 with 4 rows each (16 heads over 4 of 128): 36
// us, of 64 of 2000 in fp32 (8 over 2) 29.
#include "m3_attend_rows.h"

namespace m3 {
namespace {

// Joins rows' parts, in their order. Half a wave (a wave above headdim 128) takes a
// row's parts, or `team` of them do where there are few rows (team: a power of two).
template <typename T, Form F>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendDev a, int team) {
    __shared__ __align__(16) float o_lds[256 * 4];
    const int D = a.D, width = D <= 128 ? 32 : 64, crews = 256 / width;
    const int crew = threadIdx.x / width, lane = threadIdx.x % width, member = crew % team;
    const int64_t at = int64_t(block_id()) * (crews / team) + crew / team;
    bool live = at < a.b.tokens * a.q_heads;
    const int64_t tok = live ? at / a.q_heads : 0;
    const int head = live ? int(at - tok * a.q_heads) : 0;
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
    const int r = live ? int(t) * a.group + head % a.group : 0;
    // part p of the row lies at p0 for p = 0, at p1 + p * step beyond
    int64_t p0, p1, step;
    int parts;
    if (a.items) {
        const int e = live ? int(pair_at(a, i, r / a.rows)) : 0, rin = r % a.rows;
        const int share = a.shares[0], f = live ? a.shares[1 + e] : 0, n = live ? a.shares[2 + e] - f : 0;
        const int64_t x0 = int64_t(a.c.heads) * f + int64_t(head / a.group) * n;
        const int64_t w0 = x0 / share, w1 = (x0 + n - 1) / share;
        parts = n ? int(w1 - w0) + 1 : 0;
        live = parts > 1;  // else its workgroup wrote it (or it sees nothing)
        p0 = (2 * w0 + 1) * a.rows + rin;
        p1 = 2 * w0 * a.rows + rin;
        step = 2 * a.rows;
    } else {
        const Span sp = live ? span_of<F>(a, sq, r / a.rows * a.rows) : Span{0, 0, 0, 0};
        parts = cut_of(a, sp).pieces;
        live = live && parts > 1;
        p0 = p1 = at;
        step = a.b.tokens * a.q_heads;
    }
    if (!live) parts = 0;
    auto place = [&](int p) { return p ? p1 + p * step : p0; };
    // The first two parts of this crew are on their way while the units' maximum is found (4.4 us
    // at the least before, 3.8 since: one sequence under a window of 1024).
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

template <typename T>
void launch_join_of(const AttendDev& d, dim3 grid, int team, hipStream_t s) {
    if (d.form == kPlain) hipLaunchKernelGGL((attend_join_kernel<T, kPlain>), grid, dim3(256), 0, s, d, team);
    else hipLaunchKernelGGL((attend_join_kernel<T, kView>), grid, dim3(256), 0, s, d, team);
}
hipError_t launch_join(const AttendDev& d, m3_dtype io, hipStream_t s) {
    const JoinGrid g = join_grid(d);
    io == M3_BF16 ? launch_join_of<bf16_t>(d, g.grid, g.team, s) : launch_join_of<float>(d, g.grid, g.team, s);
    return hipGetLastError();
}
hipError_t launch_few(const AttendDev& d, m3_dtype io, hipStream_t s) {
    return d.form == kPlain ? launch_rows_form<kPlain>(d, io, s) : d.form == kView ? launch_rows_view(d, io, s)
                                                                                   : launch_rows_parts(d, io, s);
}

}  // namespace

hipError_t launch_kv_attend(const AttendArgs& a) {
    const AttendPlan& p = a.plan;
    char* ws = static_cast<char*>(a.workspace);
    auto log2_rows = [](bool packed, int rows) { return packed ? __builtin_ctz(unsigned(rows)) : 0; };
    AttendDev d{};
    d.c = a.c;
    d.b = a.b;
    d.q = a.q;
    d.out = a.out;
    d.lse = a.lse;
    d.part_o = reinterpret_cast<float*>(ws + p.o_off);
    d.part_ml = reinterpret_cast<float*>(ws + p.ml_off);
    d.shares = reinterpret_cast<int*>(ws);
    d.items = p.items;
    d.packed = log2_rows(p.packed, p.rows);
    d.q_heads = a.q_heads;
    d.group = a.q_heads / a.c.heads;
    d.D = a.c.headdim;
    d.shift = __builtin_ctz(unsigned(a.c.page_size / 16));
    d.rows = p.rows;
    d.scale2 = a.scale * kLog2e;
    d.causal = a.view.causal;
    d.window = a.view.window;
    d.row_tiles = p.row_tiles;
    d.split_tiles = p.split_tiles;
    d.splits = p.splits;
    d.wide = a.wide;
    d.blocks = p.blocks;
    d.form = p.parts ? kParts : has_view(a.view) ? kView : kPlain;
    d.view = a.view;
    d.most_prefix = int(std::min(a.view.max_prefix, ((int64_t(1) << 31) - 256) / a.c.page_size));
    hipError_t e;
    if (!p.parts) {
        if (p.tile) {
            e = launch_attend_tile(d, a.io, a.stream);
            return e != hipSuccess || p.splits == 1 ? e : launch_join(d, a.io, a.stream);
        }
        e = launch_few(d, a.io, a.stream);
        return e != hipSuccess || !p.items ? e : launch_join(d, a.io, a.stream);
    }
    const PrefixPlan& f = p.prefix;
    d.packed_a = log2_rows(f.packed, f.rows);
    d.row_tiles_a = f.row_tiles;
    d.slots = int64_t(f.slots);
    d.solo_a = int64_t(f.solo);
    d.solo_b = int64_t(f.solo_own);
    if (f.tile) {
        d.splits_a = f.splits;
        AttendDev t = d;
        t.items = 0;
        t.packed = d.packed_a;
        t.rows = f.rows;
        t.row_tiles = f.row_tiles;
        t.splits = f.splits;
        t.split_tiles = f.split_tiles;
        t.blocks = f.blocks;
        if ((e = launch_attend_tile(t, a.io, a.stream)) != hipSuccess) return e;
    } else {
        d.items_a = f.items;
    }
    if ((e = launch_few(d, a.io, a.stream)) != hipSuccess || !p.items) return e;
    return launch_merge(d, a.io, a.stream);
}

}  // namespace m3
