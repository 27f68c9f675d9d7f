// m3_kv_attend_tile.hip -- attention over the paged 8-bit cache for many rows a
// sequence (prompts, pieces of prompts).
//
// The products of m3_kv_attend.hip, S^T = K Q^T and O^T = V^T P^T with the scores
// kept in registers, but bound by the matrix rate instead of by memory: a
// workgroup of NW waves takes 16 QT NW rows, and its waves share each tile of 64
// keys, which the workgroup turns from codes into bf16 (K) and fp16 (V) once and holds in LDS.
// The LDS image is the operands themselves: a 1 KiB piece is the 64 lanes' 16
// bytes of one MFMA operand, so every read is one linear ds_read_b128 that QT
// products use. Two images alternate: the next tile's codes are on their way to
// registers while this tile is computed, and are written to the other image
// before the one barrier of a tile.
//
// The running reference is raised (and the sums scaled) only when a score passes it
// by 2^8, which fp16 still holds, so the O^T registers are mostly left alone.
#include <algorithm>

#include "m3_attend_common.h"

namespace m3 {
namespace {

template <typename T, bool FP8, int DP, int QT, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attend_tile_kernel(AttendDev a) {
    constexpr int NP = Parts<T>::kN, NV = Parts<T>::kV;
    constexpr int KM = DP / 32;          // MFMA steps of a score (32 entries each)
    constexpr int DT = DP / 16;
    constexpr int NT = 64 * NW;
    constexpr int PC = 4 * DP / NT;      // 16-code pieces of K, and of V, a thread brings
    static_assert(PC >= 1 && 4 * DP % NT == 0, "threads and pieces");
    constexpr int KB = 64 * DP * 2;      // bytes of K's, and of V's, image
    extern __shared__ __align__(16) char lds[];  // [2][K image, V image]
    __shared__ float sc_lds[2][4][4];    // of the tile's blocks: K scale, log2 and inverse of V's, whether held

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, g = lane >> 4;
    // Workgroups go to the 8 XCDs in turn; each XCD gets a run of neighbours, which
    // read the same keys of one (sequence, head, split) through its L2 at one time.
    int64_t id = (blockIdx.x & 7) * int64_t(gridDim.x / 8) + (blockIdx.x >> 3);
    if (id >= a.blocks) return;
    const int64_t rt = a.row_tiles - 1 - id % a.row_tiles;  // causal: the longest first
    id /= a.row_tiles;
    const int split = int(id % a.splits);
    id /= a.splits;
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
        if (t0 >= t1) return;
    }
    const int64_t held = min(int64_t(sq.held), a.b.max_kv);
    const int D = a.D;

    // this wave's rows
    u32x4 qf[QT][KM][NP];
    int klo[QT], khi[QT];
    int w_lo = 0x7fffffff, w_hi = 0, all_lo = 0, all_hi = 0x7fffffff;
    const int wr0 = r0 + wave * 16 * QT;
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int r = wr0 + 16 * qt + lr;
        const bool live = r < rows;
        const int tok = live ? r / a.group : 0, hq = h * a.group + (live ? r % a.group : 0);
        const T* p = static_cast<const T*>(a.q.p) + (sq.row0 + tok) * a.q.token_stride + hq * a.q.head_stride;
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            const int d = 16 * (g * (KM / 2) + m / 2) + 8 * (m & 1);
#pragma unroll
            for (int k = 0; k < NP; ++k) qf[qt][m][k] = u32x4{0, 0, 0, 0};
            if (live && d < D) Parts<T>::load(p + d, a.wide, qf[qt][m]);
        }
        khi[qt] = !live ? 0 : int(min(held, a.causal ? base + tok + 1 : held));
        klo[qt] = !live || !a.window ? 0 : int(max(base + tok - a.window + 1, int64_t(0)));
        // keys that any and that every live row of the wave sees
        int lo = live ? klo[qt] : 0x7fffffff, hi = khi[qt], alo = klo[qt], ahi = live ? khi[qt] : 0x7fffffff;
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) {
            lo = min(lo, __shfl_xor(lo, x));
            hi = max(hi, __shfl_xor(hi, x));
            alo = max(alo, __shfl_xor(alo, x));
            ahi = min(ahi, __shfl_xor(ahi, x));
        }
        w_lo = min(w_lo, lo);
        w_hi = max(w_hi, hi);
        all_lo = max(all_lo, alo);
        all_hi = min(all_hi, ahi);
    }
    w_lo = __builtin_amdgcn_readfirstlane(w_lo);
    w_hi = __builtin_amdgcn_readfirstlane(w_hi);
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);

    floatx4 o[QT][DT];
    float mx[QT], sum[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        mx[qt] = -INFINITY;
        sum[qt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[qt][d] = floatx4{0, 0, 0, 0};
    }

    // what this thread brings of a tile: piece p = tid + NT j of K (16 codes of key
    // p / (DP / 16)) and of V (16 tokens of entry p % DP), both of block p / DP
    const int32_t* pages = a.b.pages + i * a.b.max_pages;
    const int64_t hoff = int64_t(h) << a.shift;
    const char* kbase = static_cast<const char*>(a.c.k);
    const char* vbase = static_cast<const char*>(a.c.v);
    u32x4 rk[PC], rv[PC];
    float rks[PC], rvs[PC];
    int64_t at[PC];
    auto find = [&](int64_t tile) {
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int64_t blk = tile * 4 + (tid + NT * j) / DP;
            at[j] = -1;
            if (tile < t1 && blk * 16 < held) {
                const int64_t b = block_at(pages, a.b.max_pages, a.c.num_pages, a.shift, H, blk);
                at[j] = b < 0 ? b : b + hoff;
            }
        }
    };
    auto fetch = [&]() {
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int p = (tid + NT * j) % DP;
            const int key = p / (DP / 16), c = p % (DP / 16);
            rk[j] = rv[j] = u32x4{0, 0, 0, 0};
            rks[j] = rvs[j] = 0.f;
            if (at[j] >= 0) {
                if (16 * c < D) rk[j] = *reinterpret_cast<const u32x4*>(kbase + (at[j] * 16 + key) * D + 16 * c);
                if (p < D) rv[j] = *reinterpret_cast<const u32x4*>(vbase + (at[j] * D + p) * 16);
                rks[j] = a.c.k_scale[at[j]];
                rvs[j] = a.c.v_scale[at[j]];
            }
        }
    };
    auto stage = [&](int64_t tile, int buf) {
        char* ki = lds + buf * 2 * KB;
        char* vi = ki + KB;
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int p = (tid + NT * j) % DP, blk = (tid + NT * j) / DP;
            const int key = p / (DP / 16), c = p % (DP / 16);
            // key 16 blk + 4 t + e is row 4 blk + e of score tile t
            const int t = key >> 2, r = 4 * blk + (key & 3);
            const int cg = c / (KM / 2), cj = c % (KM / 2);
            char* kp = ki + ((t * KM + 2 * cj) * 64 + cg * 16 + r) * 16;
            *reinterpret_cast<u32x4*>(kp) = to_bf16<FP8>(rk[j][0], rk[j][1]);
            *reinterpret_cast<u32x4*>(kp + 1024) = to_bf16<FP8>(rk[j][2], rk[j][3]);
            u32x4 v = rv[j];
            if (tile * kTile + kTile > held) {  // codes of slots that hold no token may be anything
                const int nv = int(min(max(held - (tile * kTile + 16 * blk), int64_t(0)), int64_t(16)));
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int n = min(max(nv - 4 * w, 0), 4);
                    v[w] &= n == 4 ? ~0u : (1u << (8 * n)) - 1u;
                }
            }
            char* vp = vi + ((p / 16) * 2 * 64 + blk * 16 + p % 16) * 16;
            *reinterpret_cast<u32x4*>(vp) = to_f16<FP8>(v[0], v[1]);
            *reinterpret_cast<u32x4*>(vp + 1024) = to_f16<FP8>(v[2], v[3]);
            if (p == 0) {
                const VScale vs = v_scale(rvs[j]);
                *reinterpret_cast<floatx4*>(sc_lds[buf][blk]) =
                    floatx4{rks[j] * a.scale2, vs.log2, vs.inv, at[j] >= 0 ? 1.f : 0.f};
            }
        }
    };

    if (t0 < t1) {
        find(t0);
        fetch();
        stage(t0, 0);
        find(t0 + 1);
    }
    __syncthreads();
    int buf = 0;
    for (int64_t tile = t0; tile < t1; ++tile, buf ^= 1) {
        fetch();  // tile + 1 (nothing after the last)
        const int64_t k0 = tile * kTile;
        if (k0 < w_hi && k0 + kTile > w_lo) {
            const char* ki = lds + buf * 2 * KB + lane * 16;
            const char* vi = ki + KB;
            const floatx4 sc = *reinterpret_cast<const floatx4*>(sc_lds[buf][g]);
            const float ks = sc[0], lv = sc[1], iv = sc[2];
            const bool there = sc[3] != 0.f;
            // (a scale below 0 would turn the raw maximum round: taken entry by entry)
            const bool masked = k0 < all_lo || k0 + kTile > all_hi || __any(!there || !(ks >= 0.f));
            const int key0 = int(k0) + 16 * g;

            floatx4 s[QT][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) s[qt][t] = floatx4{0, 0, 0, 0};
#pragma unroll
                for (int m = 0; m < KM; ++m) {
                    const u32x4 kf = *reinterpret_cast<const u32x4*>(ki + (t * KM + m) * 1024);
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                        for (int k = 0; k < NP; ++k) s[qt][t] = mfma(kf, qf[qt][m][k], s[qt][t]);
                }
            }
            u32x4 pf[QT][2][NV];
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                float top = -INFINITY;
                if (masked) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + 4 * t + e;
                            const float v = __builtin_fmaf(s[qt][t][e], ks, lv);
                            s[qt][t][e] = there && key >= klo[qt] && key < khi[qt] ? v : -INFINITY;
                            top = fmaxf(top, s[qt][t][e]);
                        }
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[qt][t][e]);
                    top = __builtin_fmaf(top, ks, lv);
                }
                top = quad_max(top) - kUp;
                if (__any(top > mx[qt] + kSlack)) {
                    const float m2 = fmaxf(mx[qt], top);
                    const float fade = m2 == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[qt] - m2);
                    mx[qt] = m2;
                    sum[qt] *= fade;
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[qt][d] *= fade;
                }
                const float mu = mx[qt] == -INFINITY ? 0.f : mx[qt];
                float add = 0.f;
                float p[16];
                if (masked) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = __builtin_amdgcn_exp2f(s[qt][j / 4][j % 4] - mu);
                } else {
                    const float c = lv - mu;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[qt][j / 4][j % 4], ks, c));
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) add += p[j];
                sum[qt] += add == 0.f ? 0.f : add * iv;  // (a block no row sees may hold NaN)
                pack_p<NV>(p, pf[qt]);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const u32x4 vf = *reinterpret_cast<const u32x4*>(vi + (2 * d + hf) * 1024);
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                        for (int k = 0; k < NV; ++k) o[qt][d] = mfma_f16(vf, pf[qt][hf][k], o[qt][d]);
                }
        }
        if (tile + 1 < t1) {
            stage(tile + 1, buf ^ 1);
            find(tile + 2);
        }
        __syncthreads();
    }

#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const float l = quad_sum(sum[qt]);
        const int r = wr0 + 16 * qt + lr;
        if (r >= rows) continue;
        const int64_t row = (sq.row0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
        const bool whole = a.splits == 1;
        const float f = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const int64_t pt = whole ? row : split * a.b.tokens * a.q_heads + row;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            if (16 * d >= D) break;
            const floatx4 v = o[qt][d] * f;
            const int64_t e = pt * D + 16 * d + 4 * g;
            if (!whole) {
                *reinterpret_cast<floatx4*>(a.part_o + e) = v;
            } else if constexpr (NP == 1) {
                *reinterpret_cast<u32x2*>(static_cast<T*>(a.out) + e) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            } else {
                *reinterpret_cast<floatx4*>(static_cast<T*>(a.out) + e) = v;
            }
        }
        if (g == 0) {
            if (!whole)
                *reinterpret_cast<float2*>(a.part_ml + 2 * pt) = float2{mx[qt], l};
            else if (a.lse)
                a.lse[row] = l == 0.f ? -INFINITY : mx[qt] * kLn2 + __logf(l);
        }
    }
}

template <typename T, bool FP8, int DP, int QT, int NW>
hipError_t launch_one(const AttendDev& d, hipStream_t s) {
    constexpr int kLds = 4 * 64 * DP * 2;
    hipLaunchKernelGGL((attend_tile_kernel<T, FP8, DP, QT, NW>), dim3(unsigned((d.blocks + 7) / 8 * 8)), dim3(64 * NW),
                       kLds, s, d);
    return hipGetLastError();
}
template <typename T, bool FP8>
hipError_t launch_io(const AttendDev& d, hipStream_t s) {
    if (d.D <= 64) return launch_one<T, FP8, 64, 2, 4>(d, s);
    return launch_one<T, FP8, 128, 2, 8>(d, s);
}

}  // namespace

hipError_t launch_attend_tile(const AttendDev& d, hipStream_t s) {
    return d.c.format == M3_KV_FP8 ? launch_io<bf16_t, true>(d, s) : launch_io<bf16_t, false>(d, s);
}

}  // namespace m3
