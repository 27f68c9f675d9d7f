// m3_kv_attend.hip -- softmax attention over the paged 8-bit cache.
//
// o = sum_j p_j v_j with p the softmax of scale * q . k_j, in one pass over the
// keys with the running maximum m and sum l (log2 domain): when m grows, what
// was summed is scaled by 2^(m_old - m_new). The codes are exact in bf16, so
// both products run on bf16 MFMA with the block scales applied to the fp32
// scores (K) and to the probabilities (V); fp32 rows are split into three bf16
// parts (24 bits), which keeps every product exact.
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

#include "m3_attn_device.h"
#include "m3_attn_internal.h"

namespace m3 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;  // keys of a tile
constexpr int kWaves = 4;

struct AttendDev {
    m3_kv_cache c;
    m3_kv_batch b;
    m3_rows q;
    void* out;
    float* lse;
    float* part_o;   // [splits][tokens][q_heads][D], sums relative to the part's maximum
    float* part_ml;  // [splits][tokens][q_heads][2], maximum (log2) and sum
    int q_heads, group, D, shift, rows;
    float scale2;    // scale * log2(e)
    int causal;
    int64_t window, row_tiles, split_tiles;
    int splits;
    bool wide;
};

__device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// Tiles of 64 keys that rows r0 .. r0 + rows - 1 of a sequence can see.
struct Span {
    int64_t lo, hi;
};
__device__ __forceinline__ Span span_of(const AttendDev& a, const Seq& s, int r0) {
    const int r1 = min(r0 + a.rows, s.n * a.group) - 1;
    const int64_t base = int64_t(s.held) - s.n;
    int64_t hi = min(int64_t(s.held), a.b.max_kv), lo = 0;
    if (a.causal) hi = min(hi, base + r1 / a.group + 1);
    if (a.window) lo = max(int64_t(0), base + r0 / a.group - a.window + 1);
    if (hi <= lo) return Span{0, 0};
    return Span{lo / kTile, (hi + kTile - 1) / kTile};
}

// 8 entries of a query row as MFMA operands: one bf16 part, or three that add
// up to the fp32 value.
template <typename T>
struct Parts;
template <>
struct Parts<bf16_t> {
    static constexpr int kN = 1;
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

template <bool FP8>
__device__ __forceinline__ u32x4 to_bf16(unsigned a, unsigned b) {
    const u32x2 x = Code<FP8>::dec4_bf16(a), y = Code<FP8>::dec4_bf16(b);
    return u32x4{x[0], x[1], y[0], y[1]};
}

template <typename T, bool FP8, int DP, int QT>
__global__ __launch_bounds__(64 * kWaves) void attend_rows_kernel(AttendDev a) {
    constexpr int NP = Parts<T>::kN;   // bf16 parts of a query or probability
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
    int64_t t0 = sp.lo, t1 = sp.hi;
    if (a.splits > 1) {
        t0 = sp.lo + split * a.split_tiles;
        t1 = min(sp.hi, t0 + a.split_tiles);
        if (t0 >= t1) return;  // no such part: the join counts the same parts
    }

    // the rows' operands and the keys that each row sees
    u32x4 qf[QT][2 * KC][NP];
    int64_t klo[QT], khi[QT];
    const int D = a.D;
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
        khi[qt] = !live ? 0 : min(min(int64_t(sq.held), a.b.max_kv), a.causal ? base + tok + 1 : INT64_MAX);
        klo[qt] = a.window ? base + tok - a.window + 1 : 0;
    }
    // keys that every row sees: tiles inside need no mask
    const int rl = min(r0 + a.rows, rows) - 1;
    const int64_t held = min(int64_t(sq.held), a.b.max_kv);
    const int64_t all_hi = a.causal ? min(held, base + r0 / a.group + 1) : held;
    const int64_t all_lo = a.window ? base + rl / a.group - a.window + 1 : 0;

    const int32_t* pages = a.b.pages + i * a.b.max_pages;
    const int64_t hoff = int64_t(h) << a.shift;
    auto find = [&](int64_t blk) -> int64_t {  // its index for this head, -1: none
        if (blk * 16 >= held) return -1;
        const int64_t at = block_at(pages, a.b.max_pages, a.c.num_pages, a.shift, H, blk);
        return at < 0 ? at : at + hoff;
    };
    const char* kbase = static_cast<const char*>(a.c.k);
    const char* vbase = static_cast<const char*>(a.c.v);

    floatx4 o[QT][DT];
    float mx[QT], sum[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        mx[qt] = -INFINITY;
        sum[qt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[qt][d] = floatx4{0, 0, 0, 0};
    }

    u32x4 kr[4][KC];
    auto load_k = [&](int64_t kb) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                const int c = g * KC + j;
                kr[t][j] = u32x4{0, 0, 0, 0};
                if (kb >= 0 && 16 * c < D)
                    kr[t][j] = *reinterpret_cast<const u32x4*>(kbase + (kb * 16 + 4 * t + (lr & 3)) * D + 16 * c);
            }
    };
    int64_t tile = t0 + wave;
    int64_t kb = -1, vb = -1;
    if (tile < t1) {
        kb = find(tile * 4 + (lr >> 2));
        vb = find(tile * 4 + g);
        load_k(kb);
    }
    for (; tile < t1; tile += kWaves) {
        u32x4 vr[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            vr[d] = u32x4{0, 0, 0, 0};
            if (vb >= 0 && 16 * d < D)
                vr[d] = *reinterpret_cast<const u32x4*>(vbase + (vb * D + 16 * d + lr) * 16);
        }
        const float ks = (vb >= 0 ? a.c.k_scale[vb] : 0.f) * a.scale2;
        const float vs = vb >= 0 ? a.c.v_scale[vb] : 0.f;
        const bool there = vb >= 0;
        const int64_t key0 = tile * kTile + 16 * g;
        const bool masked = tile * kTile < all_lo || tile * kTile + kTile > all_hi || __any(!there);
        const int64_t next = tile + kWaves;
        int64_t kb2 = -1, vb2 = -1;
        if (next < t1) {
            kb2 = find(next * 4 + (lr >> 2));
            vb2 = find(next * 4 + g);
        }
        if (masked) {  // codes of slots that hold no token may be anything
            const int nv = int(min(max(held - key0, int64_t(0)), int64_t(16)));
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int n = min(max(nv - 4 * w, 0), 4);
                const unsigned keep = n == 4 ? ~0u : (1u << (8 * n)) - 1u;
#pragma unroll
                for (int d = 0; d < DT; ++d) vr[d][w] &= keep;
            }
        }

        floatx4 s[QT][4];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt)
#pragma unroll
            for (int t = 0; t < 4; ++t) s[qt][t] = floatx4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int m = 0; m < 2 * KC; ++m) {
                const u32x4 kf = to_bf16<FP8>(kr[t][m / 2][2 * (m & 1)], kr[t][m / 2][2 * (m & 1) + 1]);
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int k = 0; k < NP; ++k) s[qt][t] = mfma(kf, qf[qt][m][k], s[qt][t]);
            }
        if (next < t1) load_k(kb2);

        u32x4 pf[QT][2][NP];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = s[qt][t][e] * ks;
                    if (masked) {
                        const int64_t key = key0 + 4 * t + e;
                        v = there && key >= klo[qt] && key < khi[qt] ? v : -INFINITY;
                    }
                    s[qt][t][e] = v;
                    top = fmaxf(top, v);
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m2 = fmaxf(mx[qt], top);
            const float mu = m2 == -INFINITY ? 0.f : m2;  // nothing seen yet: 2^-inf = 0 below
            const float fade = __builtin_amdgcn_exp2f(mx[qt] - mu);
            mx[qt] = m2;
            float add = 0.f;
            float p[16];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w = __builtin_amdgcn_exp2f(s[qt][t][e] - mu);
                    add += w;
                    // (a masked key's scale may be NaN)
                    p[4 * t + e] = masked && s[qt][t][e] == -INFINITY ? 0.f : w * vs;
                }
            sum[qt] = sum[qt] * fade + add;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[qt][d] *= fade;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    if constexpr (NP == 1) {
                        pf[qt][hf][0][w] = pack_bf16(p[8 * hf + 2 * w], p[8 * hf + 2 * w + 1]);
                    } else {
                        unsigned u[3];
                        split3(p[8 * hf + 2 * w], p[8 * hf + 2 * w + 1], u);
#pragma unroll
                        for (int k = 0; k < NP; ++k) pf[qt][hf][k][w] = u[k];
                    }
                }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const u32x4 vf = to_bf16<FP8>(vr[d][2 * hf], vr[d][2 * hf + 1]);
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int k = 0; k < NP; ++k) o[qt][d] = mfma(vf, pf[qt][hf][k], o[qt][d]);
            }
        kb = kb2;
        vb = vb2;
    }

    // the four waves' sums, brought to one maximum and added
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        sum[qt] += __shfl_xor(sum[qt], 16);
        sum[qt] += __shfl_xor(sum[qt], 32);
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
void launch_rows(const AttendDev& d, int64_t blocks, hipStream_t s) {
    hipLaunchKernelGGL((attend_rows_kernel<T, FP8, DP, QT>), dim3(unsigned(blocks)), dim3(64 * kWaves), 0, s, d);
}
template <typename T, bool FP8>
hipError_t launch_attend(const AttendArgs& a) {
    const AttendPlan& p = a.plan;
    char* ws = static_cast<char*>(a.workspace);
    AttendDev d{a.c, a.b, a.q, a.out, a.lse, reinterpret_cast<float*>(ws + p.o_off),
                reinterpret_cast<float*>(ws + p.ml_off), a.q_heads, a.q_heads / a.c.heads, a.c.headdim,
                __builtin_ctz(unsigned(a.c.page_size / 16)), p.rows, a.scale * kLog2e, a.causal, a.window, p.row_tiles,
                p.split_tiles, p.splits, a.wide};
    const int64_t blocks = a.b.batch * a.c.heads * p.row_tiles * p.splits;
    const int qt = p.rows / 16, dp = d.D <= 64 ? 64 : d.D <= 128 ? 128 : 256;
    if (dp == 64) {
        if (qt == 1) launch_rows<T, FP8, 64, 1>(d, blocks, a.stream);
        else launch_rows<T, FP8, 64, 2>(d, blocks, a.stream);
    } else if (dp == 128) {
        if (qt == 1) launch_rows<T, FP8, 128, 1>(d, blocks, a.stream);
        else launch_rows<T, FP8, 128, 2>(d, blocks, a.stream);
    } else {
        launch_rows<T, FP8, 256, 1>(d, blocks, a.stream);
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
