// m3_kv_attend.hip -- softmax attention over the paged 8-bit cache.
//
// o = sum_j p_j v_j with p the softmax of scale * q . k_j, in one pass over the
// keys with a running reference and sum (log2 domain): when the reference grows,
// what was summed is scaled down. The codes are exact in bf16 and fp16, so the
// products run on MFMA over the codes themselves, q . k in bf16 and p . v in fp16,
// with the block scales applied in fp32: K's to the scores, V's as log2 vs in the
// probabilities' exponents (pack_p's comment). fp32 rows are split into three bf16
// parts (24 bits) and their probabilities into two fp16 parts, so that nothing is
// rounded to fewer bits.
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
#include <algorithm>

#include "m3_attend_common.h"

namespace m3 {
namespace {

constexpr int kWaves = 4;

// Keeps what is computed from a register after this point, where the compiler would
// convert a tile's codes early and hold them at twice or four times their size.
__device__ __forceinline__ unsigned here(unsigned w) {
    asm volatile("" : "+v"(w));
    return w;
}

// FULL: headdim is DP, so that every piece is there and loads have constant offsets.
template <typename T, bool FP8, int DP, int QT, bool FULL>
__global__ __launch_bounds__(64 * kWaves, DP == 256 || (sizeof(T) == 4 && DP * QT > 128) ? 1 : 2) void attend_rows_kernel(AttendDev a) {
    constexpr int NP = Parts<T>::kN, NV = Parts<T>::kV;
    constexpr int KC = DP / 64;        // 16-code pieces of a key row a lane holds
    constexpr int DT = DP / 16;        // 16-entry tiles of the output
    constexpr int OS = DP + 4;         // LDS row of a wave's output
    __shared__ __align__(16) float o_lds[kWaves][16][OS];
    __shared__ float m_lds[kWaves][16 * QT], l_lds[kWaves][16 * QT];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane & 15, g = lane >> 4;
    int64_t id = blockIdx.x;
    const int split = int(id % a.splits);
    id /= a.splits;
    const int64_t rt = id % a.row_tiles;
    id /= a.row_tiles;
    const int H = a.c.heads, h = int(id % H);
    const int64_t i = id / H;
    const Seq sq = seq_of(a.b, i);
    const int rows = sq.n * a.group;
    if (rt * a.rows >= rows) return;
    const int r0 = int(rt) * a.rows;
    const int64_t base = int64_t(sq.held) - sq.n;
    const Span sp = span_of(a, sq, r0);
    int t0 = int(sp.lo), t1 = int(sp.hi);
    if (a.splits > 1) {
        t0 = int(min(sp.lo + split * a.split_tiles, sp.hi));
        t1 = int(min(sp.hi, t0 + a.split_tiles));
        if (t0 >= t1) return;  // no such part: the join counts the same parts
    }
    if (a.c.num_pages == 0) t1 = t0;

    const int D = FULL ? DP : a.D;
    const int held = int(min(int64_t(sq.held), a.b.max_kv)), held_blocks = (held + 15) / 16;
    const int32_t* pages = a.b.pages + i * a.b.max_pages;
    auto find = [&](int blk) {  // a block's index for this head, -1: none (there are fewer than 2^31)
        if (blk >= held_blocks || (blk >> a.shift) >= a.b.max_pages) return -1;
        const int64_t p = pages[blk >> a.shift];
        if (p < 0 || p >= a.c.num_pages) return -1;
        return ((int(p) * H + h) << a.shift) + (blk & ((1 << a.shift) - 1));
    };
    // Loads are unconditional (of block 0 where there is none, of piece 0 beyond
    // headdim): a load behind a branch would wait for those before it. What they bring
    // is masked below, or meets zeros of q.
    const char* kbase = static_cast<const char*>(a.c.k) + (lr & 3) * D + (FULL ? 16 * g * KC : 0);
    const char* vbase = static_cast<const char*>(a.c.v) + lr * 16;
    u32x4 kr[4][KC];
    auto load_k = [&](int kb) {
        const char* p = kbase + uint64_t(unsigned(max(kb, 0))) * unsigned(16 * D);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                const int c = g * KC + j;
                kr[t][j] = *reinterpret_cast<const u32x4*>(p + 4 * t * D + (FULL ? 16 * j : 16 * c < D ? 16 * c : 0));
            }
    };
    int tile = t0 + wave;
    int kb = -1, vb = -1;
    if (tile < t1) {
        kb = find(tile * 4 + (lr >> 2));
        vb = find(tile * 4 + g);
        load_k(kb);
    }

    // the rows' operands and the keys that each row sees
    u32x4 qf[QT][2 * KC][NP];
    int klo[QT], khi[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int r = r0 + 16 * qt + lr;
        const bool live = r < rows;
        const int tok = live ? r / a.group : 0, hq = h * a.group + (live ? r % a.group : 0);
        const T* p = static_cast<const T*>(a.q.p) + (sq.row0 + tok) * a.q.token_stride + hq * a.q.head_stride;
#pragma unroll
        for (int m = 0; m < 2 * KC; ++m) {
            const int d = 16 * (g * KC + m / 2) + 8 * (m & 1);
#pragma unroll
            for (int k = 0; k < NP; ++k) qf[qt][m][k] = u32x4{0, 0, 0, 0};
            if (live && d < D) Parts<T>::load(p + d, a.wide, qf[qt][m]);
        }
        khi[qt] = !live ? 0 : a.causal ? int(min(int64_t(held), base + tok + 1)) : held;
        klo[qt] = !live || !a.window ? 0 : int(max(base + tok - a.window + 1, int64_t(0)));
    }
    // keys that every row sees: tiles inside need no mask
    const int rl = min(r0 + a.rows, rows) - 1;
    const int all_hi = a.causal ? int(max(min(int64_t(held), base + r0 / a.group + 1), int64_t(0))) : held;
    const int all_lo = a.window ? int(max(base + rl / a.group - a.window + 1, int64_t(0))) : 0;

    floatx4 o[QT][DT];
    float mx[QT], sum[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        mx[qt] = -INFINITY;
        sum[qt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[qt][d] = floatx4{0, 0, 0, 0};
    }
    for (; tile < t1; tile += kWaves) {
        u32x4 vr[DT];
        {
            const char* p = vbase + uint64_t(unsigned(max(vb, 0))) * unsigned(16 * D);
#pragma unroll
            for (int d = 0; d < DT; ++d)
                vr[d] = *reinterpret_cast<const u32x4*>(p + (FULL || 16 * d < D ? 256 * d : 0));
        }
        const bool there = vb >= 0;
        float ks = a.c.k_scale[max(vb, 0)] * a.scale2;
        VScale vs = v_scale(a.c.v_scale[max(vb, 0)]);
        const int k0 = tile * kTile, next = tile + kWaves;
        int kb2 = -1, vb2 = -1;
        if (next < t1) {
            kb2 = find(next * 4 + (lr >> 2));
            vb2 = find(next * 4 + g);
        }

        floatx4 s[QT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int m = 0; m < 2 * KC; ++m) {
                const u32x4 kf = to_bf16<FP8>(here(kr[t][m / 2][2 * (m & 1)]), here(kr[t][m / 2][2 * (m & 1) + 1]));
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
                    if (m == 0) s[qt][t] = floatx4{0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < NP; ++k) s[qt][t] = mfma(kf, qf[qt][m][k], s[qt][t]);
                }
                if (m % 4 == 3 || m == 2 * KC - 1) __builtin_amdgcn_sched_barrier(0);  // (conversions one after the other)
            }
        if (next < t1) load_k(kb2);

        // (a scale below 0 would turn the raw maximum round)
        if (k0 < all_lo || k0 + kTile > all_hi || __any(!there || !(ks >= 0.f))) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int key = k0 + 16 * g + j;
                    const float v = __builtin_fmaf(s[qt][j / 4][j % 4], ks, vs.log2);
                    s[qt][j / 4][j % 4] = there && key >= klo[qt] && key < khi[qt] ? v : -INFINITY;
                }
            ks = 1.f;
            vs.log2 = 0.f;
            // codes of slots that hold no token may be anything
            const int nv = there ? min(max(held - (k0 + 16 * g), 0), 16) : 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int n = min(max(nv - 4 * w, 0), 4);
                const unsigned keep = n == 4 ? ~0u : (1u << (8 * n)) - 1u;
#pragma unroll
                for (int d = 0; d < DT; ++d) vr[d][w] &= keep;
            }
        }
        float c[QT];
        bool up = false;
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float top = s[qt][0][0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top = fmaxf(top, s[qt][j / 4][j % 4]);
            c[qt] = quad_max(__builtin_fmaf(top, ks, vs.log2)) - kUp;
            up |= c[qt] > mx[qt] + kSlack;
        }
        if (__any(up)) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                const float m2 = fmaxf(mx[qt], c[qt]);
                const float fade = m2 == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[qt] - m2);
                mx[qt] = m2;
                sum[qt] *= fade;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[qt][d] *= fade;
            }
        }
        u32x4 pf[QT][2][NV];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            const float off = vs.log2 - (mx[qt] == -INFINITY ? 0.f : mx[qt]);
            float add = 0.f;
            float p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[qt][j / 4][j % 4], ks, off));
                add += p[j];
            }
            sum[qt] += add == 0.f ? 0.f : add * vs.inv;  // (a block no row sees may hold NaN)
            pack_p<NV>(p, pf[qt]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const u32x4 vf = to_f16<FP8>(here(vr[d][2 * hf]), here(vr[d][2 * hf + 1]));
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int k = 0; k < NV; ++k) o[qt][d] = mfma_f16(vf, pf[qt][hf][k], o[qt][d]);
                if (hf && d % 2) __builtin_amdgcn_sched_barrier(0);
            }
        kb = kb2;
        vb = vb2;
    }

    // the four waves' sums, brought to one maximum and added
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        sum[qt] = quad_sum(sum[qt]);
        if (g == 0) {
            m_lds[wave][16 * qt + lr] = mx[qt];
            l_lds[wave][16 * qt + lr] = sum[qt];
        }
    }
    __syncthreads();
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        float m = m_lds[0][16 * qt + lr];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, m_lds[w][16 * qt + lr]);
        const float f = mx[qt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[qt] - m);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<floatx4*>(&o_lds[wave][lr][16 * d + 4 * g]) = o[qt][d] * f;
        __syncthreads();
        const int per = D / 8;
        for (int e = threadIdx.x; e < 16 * per; e += 64 * kWaves) {
            const int q = e / per, d = 8 * (e - q * per);
            const int r = r0 + 16 * qt + q;
            if (16 * qt + q >= a.rows || r >= rows) continue;
            float mm = m_lds[0][16 * qt + q];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, m_lds[w][16 * qt + q]);
            float l = 0.f, v[8] = {};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float mw = m_lds[w][16 * qt + q];
                l += mw == -INFINITY ? l_lds[w][16 * qt + q] : l_lds[w][16 * qt + q] * __builtin_amdgcn_exp2f(mw - mm);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += o_lds[w][q][d + k];
            }
            const int64_t at = (sq.row0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
            if (a.splits == 1) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= inv;
                store8<true>(static_cast<T*>(a.out) + at * D + d, v);
                if (a.lse && d == 0) a.lse[at] = l == 0.f ? -INFINITY : mm * kLn2 + __logf(l);
            } else {
                const int64_t pt = split * a.b.tokens * a.q_heads + at;
                store8<true>(a.part_o + pt * D + d, v);
                if (d == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * pt) = float2{mm, l};
            }
        }
        __syncthreads();
    }
}

// Joins a row's parts, in order: one workgroup a (token, head).
template <typename T>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendDev a) {
    __shared__ float o_lds[4][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t at = blockIdx.x;
    const int64_t tok = at / a.q_heads;
    const int head = int(at - tok * a.q_heads);
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
    if (t < 0 || t >= sq.n) return;
    const int r = int(t) * a.group + head % a.group;
    const Span sp = span_of(a, sq, r / a.rows * a.rows);
    const int parts = int((sp.hi - sp.lo + a.split_tiles - 1) / a.split_tiles);
    const int64_t step = a.b.tokens * a.q_heads;
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 64) m = fmaxf(m, a.part_ml[2 * (p * step + at)]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    float l = 0.f;
    for (int p = lane; p < parts; p += 64) {
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * (p * step + at));
        l += ml.x == -INFINITY ? ml.y : ml.y * __builtin_amdgcn_exp2f(ml.x - m);
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
    const int D = a.D;
    floatx4 v{0, 0, 0, 0};
    if (4 * lane < D) {
#pragma unroll 4
        for (int p = wave; p < parts; p += 4) {
            const float mp = a.part_ml[2 * (p * step + at)];
            const float f = mp == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mp - m);
            v += *reinterpret_cast<const floatx4*>(a.part_o + (p * step + at) * D + 4 * lane) * f;
        }
        *reinterpret_cast<floatx4*>(&o_lds[wave][4 * lane]) = v;
    }
    __syncthreads();
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int d = threadIdx.x; d < D; d += 256)
        Io<T>::store(static_cast<T*>(a.out), at * D + d, (o_lds[0][d] + o_lds[1][d] + o_lds[2][d] + o_lds[3][d]) * inv);
    if (a.lse && threadIdx.x == 0) a.lse[at] = l == 0.f ? -INFINITY : m * kLn2 + __logf(l);
}

template <typename T, bool FP8, int DP, int QT>
void launch_rows(const AttendDev& d, hipStream_t s) {
    const dim3 grid(unsigned(d.blocks)), block(64 * kWaves);
    if (d.D == DP)
        hipLaunchKernelGGL((attend_rows_kernel<T, FP8, DP, QT, true>), grid, block, 0, s, d);
    else
        hipLaunchKernelGGL((attend_rows_kernel<T, FP8, DP, QT, false>), grid, block, 0, s, d);
}
template <typename T, bool FP8>
hipError_t launch_attend(const AttendArgs& a) {
    const AttendPlan& p = a.plan;
    char* ws = static_cast<char*>(a.workspace);
    AttendDev d{a.c, a.b, a.q, a.out, a.lse, reinterpret_cast<float*>(ws + p.o_off),
                reinterpret_cast<float*>(ws + p.ml_off), a.q_heads, a.q_heads / a.c.heads, a.c.headdim,
                __builtin_ctz(unsigned(a.c.page_size / 16)), p.rows, a.scale * kLog2e, a.causal, a.window, p.row_tiles,
                p.split_tiles, p.splits, a.wide, a.b.batch * a.c.heads * p.row_tiles * p.splits};
    if (p.tile) {
        hipError_t e = launch_attend_tile(d, a.io, a.stream);
        if (e != hipSuccess || p.splits == 1) return e;
        hipLaunchKernelGGL((attend_join_kernel<T>), dim3(unsigned(a.b.tokens * a.q_heads)), dim3(256), 0, a.stream, d);
        return hipGetLastError();
    }
    const int qt = p.rows / 16, dp = d.D <= 64 ? 64 : d.D <= 128 ? 128 : 256;
    if (dp == 64) {
        if (qt == 1) launch_rows<T, FP8, 64, 1>(d, a.stream);
        else launch_rows<T, FP8, 64, 2>(d, a.stream);
    } else if (dp == 128) {
        if (qt == 1) launch_rows<T, FP8, 128, 1>(d, a.stream);
        else launch_rows<T, FP8, 128, 2>(d, a.stream);
    } else {
        launch_rows<T, FP8, 256, 1>(d, a.stream);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((attend_join_kernel<T>), dim3(unsigned(a.b.tokens * a.q_heads)), dim3(256), 0, a.stream, d);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_attend(const AttendArgs& a) {
    const bool fp8 = a.c.format == M3_KV_FP8;
    if (a.io == M3_BF16) return fp8 ? launch_attend<bf16_t, true>(a) : launch_attend<bf16_t, false>(a);
    return fp8 ? launch_attend<float, true>(a) : launch_attend<float, false>(a);
}

}  // namespace m3
