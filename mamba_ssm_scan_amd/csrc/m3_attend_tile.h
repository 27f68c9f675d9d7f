// m3_attend_tile.h -- the attention kernel for many rows a sequence, as
// m3_kv_attend_tile.hip describes it, in its three forms (kPlain, kView, kParts).
// Device code only.
#pragma once
#include <algorithm>

#include "m3_attend_common.h"

namespace m3 {
namespace {

template <typename T, bool FP8, int DP, int QT, int NW, Form F>
__global__ __launch_bounds__(64 * NW, DP == 64 && !(F == kView && QT == 2) ? 3 : 2) void attend_tile_kernel(AttendDev a) {
    constexpr int NP = Parts<T>::kN, NV = Parts<T>::kV;
    constexpr int KM = DP / 32;          // MFMA steps of a score (32 entries each)
    constexpr int DT = DP / 16;
    constexpr int NT = 64 * NW;
    constexpr int PC = 4 * DP / NT;      // 16-code pieces of K, and of V, a thread brings
    static_assert(PC >= 1 && 4 * DP % NT == 0, "threads and pieces");
    constexpr bool kAhead = DP == 128;
    constexpr int KB = 64 * DP * 2;      // bytes of K's, and of V's, image
    extern __shared__ __align__(16) char lds[];  // two K images, two V images
    __shared__ float sc_lds[2][4][4];    // of the tile's blocks: K scale, log2 and inverse of V's, whether held

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, g = lane >> 4;
    // Workgroups go to the 8 XCDs in turn. A column is the row tiles of one (sequence,
    // head, split), which read the same keys; each XCD takes whole columns, a.columns of
    // them side by side, the last row tiles (with a causal mask the longest) of all first.
    // Where that would leave XCDs idle (0), every XCD takes row tiles of all columns.
    const int wg = int(block_id());
    if (wg >= a.grid) return;
    const int H = a.c.heads;
    int64_t id, rt;
    if (a.packed) {  // (later row tiles, with a causal mask the longer, first)
        const int each = H * a.splits;
        const int e = (int(a.blocks) - 1 - wg) / each;
        const Unit u = F == kParts ? group_pair_of(a, e) : pair_of(a, e);
        rt = u.at;
        id = u.i * each + wg % each;
    } else if (a.columns) {
        const int x = wg & 7, l = wg >> 3;
        const int mine = int((a.blocks / a.row_tiles - x + 7) / 8);  // columns of this XCD
        const int at = l / int(a.columns * a.row_tiles), in = l % int(a.columns * a.row_tiles);
        const int beside = min(a.columns, mine - at * a.columns);
        if (beside <= 0 || in >= beside * a.row_tiles) return;
        rt = a.row_tiles - 1 - in / beside;
        id = (at * a.columns + in % beside) * int64_t(8) + x;
    } else {
        const int64_t all = a.blocks / a.row_tiles;
        rt = a.row_tiles - 1 - wg / all;
        id = wg % all;
    }
    const int split = int(id % a.splits);
    id /= a.splits;
    const int h = int(id % H);
    const int64_t i = id / H;
    Seq sq;
    Group gr{};
    if constexpr (F == kParts) {  // a group's rows over its prefix
        gr = group_at(a, i);
        sq = Seq{gr.row0, gr.n, gr.held, 0};
    } else {
        sq = seq_of(a.b, i);
    }
    const int rows = sq.n * a.group;
    if (rt < 0 || rt * a.rows >= rows) return;
    const int r0 = int(rt) * a.rows;
    const int64_t base = sq.base;
    const Span sp = F == kParts ? Span{0, (gr.held + kTile - 1) / kTile, 0, 0} : span_of<F>(a, sq, r0);
    int t0 = int(sp.lo), t1 = int(sp.hi);
    bool whole = F != kParts;
    if (a.splits > 1) {
        const Cut cut = F == kParts ? cut_of(int(sp.hi), a.splits, kPrefixPiece) : cut_of(a, sp);
        if (split >= cut.pieces) return;
        whole = F != kParts && cut.pieces == 1;
        t0 += split * cut.per;
        t1 = min(t1, t0 + cut.per);
    }
    const int held = int(min(int64_t(sq.held), a.b.max_kv)), held_blocks = (held + 15) / 16;
    const int D = a.D;
    // of a wave's 16 keys and 4 pieces (of 16 codes) of K: this lane's
    const int key = lane & 15;  // (16 keys in turn: a group of 16 lanes writes 16 bank columns)
    auto kc = [&](int j) { return (lane >> 4) + (64 * wave + NT * j) % DP / 16; };

    // what a wave brings of a tile: piece p = 64 wave + lane + NT j of K (16 codes of a
    // key) and of V (16 tokens of entry p % DP), of block p / DP, so that a wave's
    // pieces of one j lie in one block and their page is looked up once, in scalars
    const int32_t* pages = F == kParts ? gr.pre.pages : a.b.pages + i * a.b.max_pages;
    const int swave = __builtin_amdgcn_readfirstlane(wave);
    struct Raw {
        u32x4 k[PC], v[PC];
        float ks[PC], vs[PC];
        bool there[PC];  // whether V's block (and its scales) is held
    };
    struct Pages {
        int p[PC];   // page number of this wave's blocks of a tile (-1: none)
    };
    // (kView) keys that sinks show, the first block that the window does, and the shared pages
    const int sinks = F == kView ? int(a.view.sinks) : 0, sink_blocks = (sinks + 15) / 16;
    const int win_block = F == kView && a.window ? int(max(base + r0 / a.group - a.window + 1, int64_t(0)) / 16) : 0;
    const Prefix pre = F == kView ? prefix_of(a, i) : Prefix{nullptr, 0};
    auto find = [&](int tile) {
        Pages r;
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int blk = tile_at<F>(sp, tile) * 4 + (64 * swave + NT * j) / DP, pg = blk >> a.shift;
            r.p[j] = -1;
            if constexpr (F == kParts) {  // (read before it is known how many entries count)
                const int p = pages[min(pg, int(a.view.max_prefix - 1))];
                if (tile < t1 && blk < held_blocks) r.p[j] = p;
                continue;
            }
            if (F == kView && blk < win_block && blk >= sink_blocks) continue;
            // (forms other than kPlain: max_kv ends in the table)
            if (tile < t1 && blk < held_blocks && (F != kPlain || pg < a.b.max_pages))
                r.p[j] = F == kView && pg < pre.count ? pre.pages[pg] : pages[pg];
        }
        return r;
    };
    auto block = [&](int tile, const Pages& pg, int j) -> int64_t {
        const int blk = tile_at<F>(sp, tile) * 4 + (64 * swave + NT * j) / DP;
        const int64_t page = __builtin_amdgcn_readfirstlane(pg.p[j]);
        if (page < 0 || page >= a.c.num_pages) return -1;
        return ((page * H + h) << a.shift) + (blk & ((1 << a.shift) - 1));
    };
    auto fetch_k = [&](Raw& r, int tile, const Pages& pg) {
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int64_t at = block(tile, pg, j);
            r.k[j] = u32x4{0, 0, 0, 0};
            if (at >= 0 && 16 * kc(j) < D)
                r.k[j] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.c.k) + at * 16 * D + key * D + 16 * kc(j));
        }
    };
    auto fetch_v = [&](Raw& r, int tile, const Pages& pg) {
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int64_t at = block(tile, pg, j);
            const int d = (64 * swave + NT * j) % DP + lane;
            r.v[j] = u32x4{0, 0, 0, 0};
            r.ks[j] = r.vs[j] = 0.f;
            r.there[j] = at >= 0;
            if (at >= 0) {
                if (d < D) r.v[j] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.c.v) + at * 16 * D + d * 16);
                r.ks[j] = a.c.k_scale[at];
                r.vs[j] = a.c.v_scale[at];
            }
        }
    };
    auto stage_k = [&](const Raw& raw, int buf) {
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int blk = (64 * swave + NT * j) / DP;
            // key 16 blk + 4 t + e is row 4 blk + e of score tile t; its place among a
            // piece's 16 rows is turned by 4 t, so that a wave's writes take all banks
            const int t = key >> 2, r = (4 * blk + (key & 3) + 4 * t) & 15;
            const int cg = kc(j) / (KM / 2), cj = kc(j) % (KM / 2);
            char* kp = lds + buf * KB + ((t * KM + 2 * cj) * 64 + cg * 16 + r) * 16;
            *reinterpret_cast<u32x4*>(kp) = to_bf16<FP8>(raw.k[j][0], raw.k[j][1]);
            *reinterpret_cast<u32x4*>(kp + 1024) = to_bf16<FP8>(raw.k[j][2], raw.k[j][3]);
        }
    };
    auto stage_v = [&](const Raw& raw, int tile, int buf) {
#pragma unroll
        for (int j = 0; j < PC; ++j) {
            const int p0 = 64 * swave + NT * j;
            const int blk = p0 / DP, d = p0 % DP + lane;
            u32x4 v = raw.v[j];
            const VScale vs = v_scale(raw.vs[j]);
            if (vs.none) v = u32x4{0, 0, 0, 0};
            const int k0 = tile_at<F>(sp, tile) * kTile;
            if (k0 + kTile > held) {  // codes of slots that hold no token may be anything
                const int nv = min(max(held - (k0 + 16 * blk), 0), 16);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int n = min(max(nv - 4 * w, 0), 4);
                    v[w] &= n == 4 ? ~0u : (1u << (8 * n)) - 1u;
                }
            }
            char* vp = lds + (2 + buf) * KB + ((d / 16) * 2 * 64 + blk * 16 + d % 16) * 16;
            *reinterpret_cast<u32x4*>(vp) = v_operand<FP8, NV>(v[0], v[1]);
            *reinterpret_cast<u32x4*>(vp + 1024) = v_operand<FP8, NV>(v[2], v[3]);
            if (p0 % DP == 0 && lane == 0) {
                *reinterpret_cast<floatx4*>(sc_lds[buf][blk]) =
                    floatx4{raw.ks[j] * a.scale2, vs.log2, vs.inv, raw.there[j] ? 1.f : 0.f};
            }
        }
    };
    // The forms other than kPlain have short runs of keys (a window's, a piece of a prefix), and
    // a wave's first waits weigh more: page numbers and the first loads go out together and
    // before the rows' own (128 steps behind 8192 tokens 1 us of 62). Each tile's loads a turn
    // earlier than in kPlain gained nothing more.
    Raw ra, rb;  // rb: the second tile's K before the loop
    Pages pgv{}, pgk{};
    if constexpr (F != kPlain) {
        if (t0 < t1) {
            const Pages first = find(t0);
            pgv = find(t0 + 1);
            pgk = find(t0 + 2);
            fetch_k(ra, t0, first);
            fetch_v(ra, t0, first);
            if constexpr (kAhead) fetch_k(rb, t0 + 1, pgv);
        }
    }

    // this wave's rows
    u32x4 qf[QT][KM][NP];
    int klo[QT], khi[QT];
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
        if constexpr (F == kParts) khi[qt] = live ? row_limit(a, gr, sq.row0 + tok) : 0;
        else khi[qt] = !live ? 0 : a.causal ? int(min(int64_t(held), base + tok + 1)) : held;
        klo[qt] = F == kParts || !live || !a.window ? 0 : int(max(base + tok - a.window + 1, int64_t(0)));
    }
    // keys that any and that every row of the wave sees (its rows follow one another)
    const int wave_rows = min(16 * QT, rows - wr0);
    const int64_t p0 = base + wr0 / a.group, p1 = base + (wr0 + wave_rows - 1) / a.group;
    int w_lo = F != kParts && a.window ? int(max(p0 - a.window + 1, int64_t(0))) : 0;
    int w_hi = wave_rows <= 0 ? 0 : a.causal ? int(max(min(int64_t(held), p1 + 1), int64_t(0))) : held;
    int all_lo = F != kParts && a.window ? int(max(p1 - a.window + 1, int64_t(0))) : 0;
    int all_hi = a.causal ? int(max(min(int64_t(held), p0 + 1), int64_t(0))) : held;
    if constexpr (F == kParts) {
        all_hi = held;
        w_hi = 0;
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            all_hi = min(all_hi, wr0 + 16 * qt + lr < rows ? khi[qt] : held);
            w_hi = max(w_hi, khi[qt]);
        }
#pragma unroll
        for (int k = 1; k < 16; k <<= 1) {
            all_hi = min(all_hi, __shfl_xor(all_hi, k));
            w_hi = max(w_hi, __shfl_xor(w_hi, k));
        }
    }
    w_lo = __builtin_amdgcn_readfirstlane(w_lo);
    w_hi = __builtin_amdgcn_readfirstlane(w_hi);
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);

    floatx4 o[QT][DT];
    float mx[QT], sum[QT], un[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        un[qt] = 1.f;
        mx[qt] = wr0 + 16 * qt + lr < rows ? -INFINITY : 0.f;
        sum[qt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[qt][d] = floatx4{0, 0, 0, 0};
    }

    // piece m of score tile t of a K image, and the scores' products with it
    int kt[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) kt[t] = g * 256 + ((lr + 4 * t) & 15) * 16;
    floatx4 s[QT][4], sn[QT][4];
    auto score_step = [&](int buf, int t, int m, floatx4 (&x)[QT][4]) {
        const u32x4 kf = *reinterpret_cast<const u32x4*>(lds + buf * KB + (t * KM + m) * 1024 + kt[t]);
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            if (m == 0) x[qt][t] = floatx4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < NP; ++k) x[qt][t] = mfma(kf, qf[qt][m][k], x[qt][t]);
        }
    };
    auto scores = [&](int buf, floatx4 (&x)[QT][4]) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int m = 0; m < KM; ++m) score_step(buf, t, m, x);
    };
    auto seen = [&](int tile) {
        const int k0 = tile_at<F>(sp, tile) * kTile;
        return k0 < w_hi && (k0 + kTile > w_lo || (F == kView && k0 < sinks));
    };

    // kAhead. In turn n the scores of tile n are in registers, V of tile n and K of tile
    // n + 1 in LDS: the products of tile n + 1's scores run beside tile n's exponentials,
    // those with V beside the conversion of what comes next (K of n + 2, V of n + 1).
    // Headdim 64 has half the products for as many exponentials: there three waves a SIMD
    // without the second set of scores do better (K and V of n + 1 are converted in turn n).
    // So do the two that headdim 256 leaves (one prompt of 2048, 16 heads over 4: bf16 103 us
    // and 108 with the second set, fp32 164 and 203, where it spills).
    if (t0 < t1) {
        if constexpr (F == kPlain) {
            pgk = find(t0);
            fetch_k(ra, t0, pgk);
            fetch_v(ra, t0, pgk);
            pgv = find(t0 + 1);
        }
        stage_k(ra, 0);
        stage_v(ra, t0, 0);
        if constexpr (kAhead) {
            if constexpr (F == kPlain) {
                fetch_k(ra, t0 + 1, pgv);
                pgk = find(t0 + 2);
                stage_k(ra, 1);
            } else {
                stage_k(rb, 1);
            }
        }
        if constexpr (kAhead) {
            __syncthreads();
            if (seen(t0)) scores(0, s);
        }
        __syncthreads();
    }
    float inv_top = -INFINITY;  // scales of a 1 / vs above it ask for the maxima (all, until every row of the wave has a reference)
    auto turn_of = [&](int tile, int buf, floatx4 (&s)[QT][4], floatx4 (&sn)[QT][4]) {
        fetch_v(ra, tile + 1, pgv);  // (nothing after the last)
        fetch_k(ra, tile + 1 + kAhead, kAhead ? pgk : pgv);
        if constexpr (kAhead) {
            pgv = pgk;
            pgk = find(tile + 3);
        } else {
            pgv = find(tile + 2);
        }
        const int k0 = tile_at<F>(sp, tile) * kTile;
        if (seen(tile)) {
            if constexpr (!kAhead) scores(buf, s);
            const floatx4 sc = *reinterpret_cast<const floatx4*>(sc_lds[buf][g]);
            float ks = sc[0], lv = sc[1];
            const float iv = sc[2];
            if ((k0 < all_lo && (F != kView || k0 + kTile > sinks)) || k0 + kTile > all_hi || __any(sc[3] == 0.f)) {
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int key = k0 + 16 * g + j;
                        const float v = __builtin_fmaf(s[qt][j / 4][j % 4], ks, lv);
                        s[qt][j / 4][j % 4] = sc[3] != 0.f && (F == kParts || key >= klo[qt] || (F == kView && key < sinks)) && key < khi[qt] ? v : -INFINITY;
                    }
                ks = 1.f;
                lv = 0.f;
            }
            u32x4 pf[QT][2][NV];
            float c[QT], add[QT];
            auto part = [&](int x) {  // probability x % 16 of row tile x / 16
                const int qt = x / 16, j = x % 16;
                return __builtin_amdgcn_exp2f(__builtin_fmaf(s[qt][j / 4][j % 4], ks, c[qt]));
            };
            auto pair = [&](int x) {
                const float lo = part(2 * x), hi = part(2 * x + 1);
                add[x / 8] = x % 8 ? add[x / 8] + lo + hi : lo + hi;
                pack_pair<NV>(lo, hi, pf[x / 8][x % 8 / 4], x % 4);
            };
            constexpr int kSteps = 4 * KM, kPairs = 8 * QT;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) c[qt] = lv - (mx[qt] == -INFINITY ? 0.f : mx[qt]);
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                if constexpr (kAhead) score_step(buf ^ 1, u / KM, u % KM, sn);
#pragma unroll
                for (int x = u * kPairs / kSteps; x < (u + 1) * kPairs / kSteps; ++x) pair(x);
            }
            bool big = false;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) big |= !(add[qt] < kF16Top);
            // From 2^15 on, before the first reference, or where a term could pass the sum's
            // range, the exact maximum is taken and all of this tile's probabilities are
            // formed again. (No short cut past `inv_top`: the arithmetic would move behind it,
            // away from the products it runs beside.)
            if (__any(int(iv > inv_top) | int(big))) {
                inv_top = kInvTop;
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 16; ++j) top = fmaxf(top, __builtin_fmaf(s[qt][j / 4][j % 4], ks, lv));
                    const float m2 = fmaxf(mx[qt], quad_max(top) - kUp);
                    const int e1 = unit_exp(un[qt]);
                    const float n2 = fmaxf(quad_max(top + __builtin_amdgcn_logf(iv)),
                                           mx[qt] - float(e1) + __builtin_amdgcn_logf(quad_sum(sum[qt])));
                    un[qt] = sum_unit(m2 - n2);
                    const float fade = m2 == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[qt] - m2);
                    sum[qt] *= m2 == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[qt] - m2 + float(unit_exp(un[qt]) - e1));
                    mx[qt] = m2;
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[qt][d] *= fade;
                    c[qt] = lv - (m2 == -INFINITY ? 0.f : m2);
#pragma unroll
                    for (int x = 0; x < 8; ++x) pair(8 * qt + x);
                    inv_top = __any(m2 == -INFINITY || un[qt] != 1.f) ? -INFINITY : inv_top;
                }
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) sum[qt] += add[qt] == 0.f ? 0.f : add[qt] * (iv * un[qt]);  // (a block no row sees may hold NaN)
            const char* vi = lds + (2 + buf) * KB + lane * 16;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const u32x4 vf = *reinterpret_cast<const u32x4*>(vi + (2 * d + hf) * 1024);
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                        for (int k = 0; k < NV; ++k) o[qt][d] = mfma_v<NV>(vf, pf[qt][hf][k], o[qt][d]);
                }
        } else if (kAhead && seen(tile + 1)) {
            scores(buf ^ 1, sn);
        }
        stage_k(ra, kAhead ? buf : buf ^ 1);
        stage_v(ra, tile + 1, buf ^ 1);
        __syncthreads();
    };
    for (int tile = t0; tile < t1; tile += 2) {
        turn_of(tile, 0, s, sn);
        if (tile + 1 < t1) {
            if constexpr (kAhead) turn_of(tile + 1, 1, sn, s);
            else turn_of(tile + 1, 1, s, sn);
        }
    }

#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const float l = quad_sum(sum[qt]);
        const int r = wr0 + 16 * qt + lr;
        if (r >= rows) continue;
        const int64_t row = (sq.row0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
        const float f = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l, unit = mx[qt] - float(unit_exp(un[qt]));
        const int64_t pt = whole ? row : split * a.b.tokens * a.q_heads + row;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            if (16 * d >= D) break;
            floatx4 v = o[qt][d] * f;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __builtin_amdgcn_ldexpf(v[k], unit_exp(un[qt]));
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
                *reinterpret_cast<float2*>(a.part_ml + 2 * pt) = float2{unit, l};
            else if (a.lse)
                a.lse[row] = l == 0.f ? -INFINITY : unit * kLn2 + __logf(l);
        }
    }
}

template <typename T, bool FP8, Form F, int DP, int QT, int NW>
hipError_t launch_one(const AttendDev& d, hipStream_t s) {
    constexpr int kLds = 4 * 64 * DP * 2;
    hipLaunchKernelGGL((attend_tile_kernel<T, FP8, DP, QT, NW, F>), grid_of(d.grid), dim3(64 * NW), kLds, s, d);
    return hipGetLastError();
}
// Rows a wave and waves (the plan's rows are their products): two tiles of 16 rows a wave where the
// registers hold them at two waves a SIMD, one where the plan halves the rows.
template <typename T, bool FP8, Form F>
hipError_t launch_io(const AttendDev& d, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (d.D <= 64) return d.rows == 64 ? launch_one<T, FP8, F, 64, 1, 4>(d, s) : launch_one<T, FP8, F, 64, 2, 4>(d, s);
        if (d.D <= 128) return d.rows == 128 ? launch_one<T, FP8, F, 128, 1, 8>(d, s) : launch_one<T, FP8, F, 128, 2, 8>(d, s);
    } else {
        if (d.D <= 64) return launch_one<T, FP8, F, 64, 1, 4>(d, s);
        if (d.D <= 128) return launch_one<T, FP8, F, 128, 1, 8>(d, s);
    }
    return launch_one<T, FP8, F, 256, 1, 8>(d, s);
}
template <Form F>
hipError_t launch_tile_form(const AttendDev& d, m3_dtype io, hipStream_t s) {
    const bool fp8 = d.c.format == M3_KV_FP8;
    if (io == M3_BF16) return fp8 ? launch_io<bf16_t, true, F>(d, s) : launch_io<bf16_t, false, F>(d, s);
    return fp8 ? launch_io<float, true, F>(d, s) : launch_io<float, false, F>(d, s);
}

}  // namespace
}  // namespace m3
