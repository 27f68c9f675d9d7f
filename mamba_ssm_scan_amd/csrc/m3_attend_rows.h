// m3_attend_rows.h -- the attention kernel for few rows a sequence, as m3_kv_attend.hip
// describes it, in its three forms (kPlain, kView, kParts). Device code only.
#pragma once
#include <algorithm>

#include "m3_attend_common.h"

namespace m3 {
namespace {

constexpr int kWaves = 4;
constexpr int kMaxItems = kAttendItems;

// (kParts) The first key of sequence i's own: behind its group's prefix.
__device__ __forceinline__ int own_key(const AttendDev& a, int64_t i) { return prefix_of(a, i).count * a.c.page_size; }

// Even shares. The tiles of all (sequence, row tile) items lie one after the other,
// an item's once for each key head; a workgroup takes the same number of them,
// whatever the lengths, and a row tile's keys that several share are joined
// afterwards. An item's keys for one head are one run: the share that holds its
// first tile but not its last writes part 0 to its slot 2 w + 1, a later share w
// the next part to slot 2 w. Every workgroup forms the items' first tiles itself
// (one scan of the lengths), the first also stores them for the join. Returns the
// tiles of a share: a multiple of 4, one tile a wave at least.
//   In the forms other than kPlain runs count a multiple of the share, their last tiles empty, so that
// a share holds one run: two short ones, one after the other, are twice the latency (about 8 us,
// where a tile more a wave is 3). There are heads * (items with keys) runs; shares of S tiles
// are enough where heads * (all / S + items with keys) <= workgroups. Where that would take 8 tiles
// more than even ones, runs count a multiple of 4 only. 18 tiles of each of 4 heads: 15 us and 10.7.
// Sums over the lanes up to each one: moves within rows of 16, then from rows before (no LDS).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // from 1, 2, 4, 8 lanes before
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of the row before, for rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31, for rows 2 and 3
    return v;
}
template <Form F>
__device__ __forceinline__ int even_shares(const AttendDev& a, int* first, int* scan) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (a.items + 64 * kWaves - 1) / (64 * kWaves);
    const int e0 = threadIdx.x * per, e1 = min(e0 + per, a.items);
    int sum = 0, held = 0;
    for (int e = e0; e < e1; ++e) {
        int n = 0;
        if (F == kParts && e < a.items_a) {
            const Unit u = group_pair_of(a, e);
            const Group gr = group_at(a, u.i);
            if (u.at >= 0 && u.at * a.rows < int64_t(gr.n) * a.group) n = (gr.held + kTile - 1) / kTile;
        } else {
            const Unit u = pair_of(a, e - (F == kParts ? a.items_a : 0));
            const Seq sq = seq_of(a.b, u.i);
            const int64_t r0 = u.at * a.rows;
            if (r0 >= 0 && r0 < sq.n * a.group) {
                const Span sp = span_of<F>(a, sq, int(r0), F == kParts ? own_key(a, u.i) : 0);
                n = int(sp.hi - sp.lo);
            }
        }
        if (F != kPlain) n = (n + 3) / 4 * 4;
        first[e] = n;
        sum += n;
        held += n > 0;
    }
    int unit = 0;  // tiles that runs count a multiple of
    if constexpr (F != kPlain) {
        const int all = wave_scan(sum), runs = wave_scan(held) * a.c.heads;
        if (lane == 63) {
            scan[wave] = all;
            scan[kWaves + wave] = runs;
        }
        __syncthreads();
        int64_t total = 0, n = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            total += scan[w];
            n += scan[kWaves + w];
        }
        total *= a.c.heads;
        const int64_t even = (total + 4 * a.blocks - 1) / (4 * a.blocks) * 4;
        if (even <= 4) {
            unit = 4;
        } else if (n < a.blocks) {
            const int64_t one = (total + 4 * (a.blocks - n) - 1) / (4 * (a.blocks - n)) * 4;
            if (one <= even + 8) unit = int(one);
        }
        if (unit > 4) {
            sum = 0;
            for (int e = e0; e < e1; ++e) {
                first[e] = (first[e] + unit - 1) / unit * unit;
                sum += first[e];
            }
        }
        __syncthreads();
    }
    const int up = wave_scan(sum);  // over the wave, then over the waves before
    if (lane == 63) scan[wave] = up;
    __syncthreads();
    int at = up - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? scan[w] : 0;
        total += scan[w];
    }
    for (int e = e0; e < e1; ++e) {
        const int n = first[e];
        first[e] = at;
        at += n;
    }
    if (threadIdx.x == 0) first[a.items] = total;
    __syncthreads();
    const int64_t all = int64_t(total) * a.c.heads;
    const int share = unit ? unit : int((all + 4 * a.blocks - 1) / (4 * a.blocks)) * 4;
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) a.shares[0] = max(share, 4);
        for (int e = threadIdx.x; e <= a.items; e += 64 * kWaves) a.shares[1 + e] = first[e];
    }
    return max(share, 4);
}
// Rows of items that see no key belong to no share: every workgroup clears its part.
template <typename T>
__device__ __forceinline__ void zero_rows(const AttendDev& a, const int* first) {
    for (int e = blockIdx.x; e < a.items; e += int(a.blocks)) {
        if (first[e + 1] != first[e]) continue;
        const Unit u = pair_of(a, e);
        const Seq sq = seq_of(a.b, u.i);
        if (u.at < 0 || u.at * a.rows >= sq.n * a.group) continue;
        const int r0 = int(u.at) * a.rows, r1 = min(r0 + a.rows, sq.n * a.group);
        const int D = a.D, H = a.c.heads;
        for (int64_t k = threadIdx.x; k < int64_t(r1 - r0) * H * D; k += 64 * kWaves) {
            const int d = int(k % D), h = int(k / D % H), r = r0 + int(k / D / H);
            const int64_t at = (sq.row0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
            Io<T>::store(static_cast<T*>(a.out), at * D + d, 0.f);
            if (a.lse && d == 0) a.lse[at] = -INFINITY;
        }
    }
}

// FULL: headdim is DP, so that every piece is there and loads have constant offsets.
// EVEN: even shares (their bookkeeping takes registers that the other case keeps for
// more waves).
// Waves a SIMD: what the registers of each case allow without spilling in its loop. (kView holds the view beside
// the rows: at headdim 128 with 32 rows one wave where kPlain has two; 64 sequences of 8 rows, 16 heads over 4,
// window 2048: 72 us with 64 sinks, 52 without.)
template <typename T, int DP, int QT, bool FULL, bool EVEN, Form F>
constexpr int kSimdWaves = DP == 256 || (sizeof(T) == 4 && DP * QT > 128)            ? 1
                           : F == kView && DP * QT > 128 && (EVEN || !FULL)          ? 1
                           : sizeof(T) == 4 || QT == 2                               ? 2
                           : DP == 64                                                ? 4
                           : EVEN || F != kPlain                                     ? 2
                                                                                     : 3;
template <typename T, bool FP8, int DP, int QT, bool FULL, bool EVEN, Form F>
__global__ __launch_bounds__(64 * kWaves, (kSimdWaves<T, DP, QT, FULL, EVEN, F>)) void attend_rows_kernel(AttendDev a) {
    constexpr int NP = Parts<T>::kN, NV = Parts<T>::kV;
    constexpr int KC = DP / 64;        // 16-code pieces of a key row a lane holds
    constexpr int DT = DP / 16;        // 16-entry tiles of the output
    constexpr int OS = DP + 4;         // LDS row of a wave's output
    __shared__ __align__(16) float o_lds[kWaves][16][OS];
    __shared__ float m_lds[kWaves][16 * QT], l_lds[kWaves][16 * QT];
    __shared__ float g_lds[kWaves][16 * QT];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane & 15, g = lane >> 4;
    const int H = a.c.heads;
    __shared__ int first_lds[EVEN ? kMaxItems + 1 : 1];
    __shared__ int scan_lds[2 * kWaves];
    const int w = int(block_id());
    if (w >= a.blocks) return;
    int64_t x = 0, xe = 1;  // what is left of this workgroup's share
    if constexpr (EVEN) {
        const int share = even_shares<F>(a, first_lds, scan_lds);
        x = int64_t(w) * share;
        xe = min(x + share, int64_t(H) * first_lds[a.items]);
        if constexpr (F != kParts) zero_rows<T>(a, first_lds);
    }
    while (x < xe) {  // (a share may end one row tile's keys and begin the next's)
        int64_t i, rt;
        int h, t0 = 0, t1 = 0;
        bool whole = true, shared = false;  // shared: a group's rows over its prefix
        if constexpr (EVEN) {
            int e = 0;
            for (int hi = a.items - 1; e < hi;) {  // the last item that begins at or before x
                const int mid = (e + hi + 1) / 2;
                if (int64_t(H) * first_lds[mid] <= x) e = mid;
                else hi = mid - 1;
            }
            e = __builtin_amdgcn_readfirstlane(e);  // (the workgroup's: in scalars)
            const int f0 = __builtin_amdgcn_readfirstlane(first_lds[e]);
            const int n = __builtin_amdgcn_readfirstlane(first_lds[e + 1]) - f0;
            const int64_t off = x - int64_t(H) * f0;
            h = int(off / n);
            t0 = int(off - int64_t(h) * n);
            t1 = int(min(int64_t(n), t0 + (xe - x)));
            x += t1 - t0;
            whole = t1 - t0 == n;
            shared = F == kParts && e < a.items_a;
            const Unit u = shared ? group_pair_of(a, e) : pair_of(a, e - (F == kParts ? a.items_a : 0));
            i = u.i;
            rt = u.at;
        } else if (a.packed) {
            x = xe;
            const Unit u = pair_of(a, w / H);
            h = w % H;
            i = u.i;
            rt = u.at;
        } else {
            x = xe;
            rt = w % a.row_tiles;
            const int64_t ih = w / a.row_tiles;
            h = int(ih % H);
            i = ih / H;
        }
        Seq sq;
        Group gr{};
        int own = 0, pieces = 0;  // (kParts) the first key of the sequence's own
        if (F == kParts && shared) {
            gr = group_at(a, i);
            sq = Seq{gr.row0, gr.n, gr.held, 0};
        } else {
            sq = seq_of(a.b, i);
            if constexpr (F == kParts) own = own_key(a, i);
            // pieces of the prefix (the kernel for many rows cut them)
            if (F == kParts && !EVEN && own > 0)
                pieces = cut_of(int((min(int64_t(own), a.b.max_kv) + kTile - 1) / kTile), a.splits_a, kPrefixPiece).pieces;
        }
        const int rows = sq.n * a.group;
        if (rt < 0 || rt * a.rows >= rows) break;  // (without shares only)
        const int r0 = int(rt) * a.rows;
        const int64_t base = sq.base;
        const Span sp = F == kParts && shared ? Span{0, (gr.held + kTile - 1) / kTile, 0, 0} : span_of<F>(a, sq, r0, own);
        const int slot = t0 > 0 ? 2 * w : 2 * w + 1;
        if constexpr (EVEN) {
            t0 += int(sp.lo);
            t1 += int(sp.lo);
            if constexpr (F != kPlain) t1 = min(t1, int(sp.hi));
        } else {
            t0 = int(sp.lo);
            t1 = int(sp.hi);
        }
        if (a.c.num_pages == 0) t1 = t0;

        const int D = FULL ? DP : a.D;
        const int held = int(min(int64_t(sq.held), a.b.max_kv)), held_blocks = (held + 15) / 16;
        // (kView) keys that sinks show, the first block that the window does, and the shared pages
        const int sinks = F == kView ? int(a.view.sinks) : 0, sink_blocks = (sinks + 15) / 16;
        const int win_block = F == kView && a.window ? int(max(base + r0 / a.group - a.window + 1, int64_t(0)) / 16) : 0;
        const Prefix pre = F == kView ? prefix_of(a, i) : Prefix{nullptr, 0};
        const int32_t* pages = F == kParts && shared ? gr.pre.pages : a.b.pages + i * a.b.max_pages;
        // (kParts) the table's end: its entries are read before it is known how many count
        const int last = F != kParts ? 0 : int((shared ? a.view.max_prefix : a.b.max_pages) - 1);
        auto find = [&](int blk) {  // a block's index for this head, -1: none (there are fewer than 2^31)
            const int pg = blk >> a.shift;
            if constexpr (F == kParts) {
                const int p = pages[min(pg, last)];
                if (blk >= held_blocks || blk < own / 16 || p < 0 || p >= a.c.num_pages) return -1;
                return ((p * H + h) << a.shift) + (blk & ((1 << a.shift) - 1));
            }
            // (forms other than kPlain: max_kv ends in the table)
            if (blk >= held_blocks || (F == kPlain && pg >= a.b.max_pages)) return -1;
            if (F == kView && blk < win_block && blk >= sink_blocks) return -1;
            const int64_t p = F == kView && pg < pre.count ? pre.pages[pg] : pages[pg];
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
        int vb = -1;
        if (tile < t1) {
            const int at = tile_at<F>(sp, tile);
            vb = find(at * 4 + g);
            load_k(find(at * 4 + (lr >> 2)));
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
            if (F == kParts && shared) khi[qt] = live ? row_limit(a, gr, sq.row0 + tok) : 0;
            else khi[qt] = !live ? 0 : a.causal ? int(min(int64_t(held), base + tok + 1)) : held;
            klo[qt] = F == kParts || !live || !a.window ? 0 : int(max(base + tok - a.window + 1, int64_t(0)));
        }
        // keys that every row sees: tiles inside need no mask
        const int rl = min(r0 + a.rows, rows) - 1;
        int all_hi = a.causal ? int(max(min(int64_t(held), base + r0 / a.group + 1), int64_t(0))) : held;
        const int all_lo = F != kParts && a.window ? int(max(base + rl / a.group - a.window + 1, int64_t(0))) : 0;
        if (F == kParts && shared) {
            all_hi = held;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) all_hi = min(all_hi, r0 + 16 * qt + lr < rows ? khi[qt] : held);
#pragma unroll
            for (int k = 1; k < 16; k <<= 1) all_hi = min(all_hi, __shfl_xor(all_hi, k));
            all_hi = __builtin_amdgcn_readfirstlane(all_hi);
        }

        floatx4 o[QT][DT];
        float mx[QT], sum[QT], un[QT];
        float inv_top = kInvTop;  // scales of a 1 / vs above it ask for the sums' units
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            mx[qt] = -INFINITY;
            sum[qt] = 0.f;
            un[qt] = 1.f;
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
            const int k0 = tile_at<F>(sp, tile) * kTile, next = tile + kWaves;
            int kb2 = -1, vb2 = -1;
            if (next < t1) {
                const int at = tile_at<F>(sp, next);
                kb2 = find(at * 4 + (lr >> 2));
                vb2 = find(at * 4 + g);
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
            if ((k0 < all_lo && (F != kView || k0 + kTile > sinks)) || k0 + kTile > all_hi || __any(!there || !(ks >= 0.f) || vs.none)) {
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int key = k0 + 16 * g + j;
                        const float x = __builtin_fmaf(s[qt][j / 4][j % 4], ks, vs.log2);
                        s[qt][j / 4][j % 4] = there && (F == kParts || key >= klo[qt] || (F == kView && key < sinks)) && key < khi[qt] ? x : -INFINITY;
                    }
                ks = 1.f;
                vs.log2 = 0.f;
                // codes of slots that hold no token may be anything
                const int nv = there && !vs.none ? min(max(held - (k0 + 16 * g), 0), 16) : 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int n = min(max(nv - 4 * w, 0), 4);
                    const unsigned keep = n == 4 ? ~0u : (1u << (8 * n)) - 1u;
#pragma unroll
                    for (int d = 0; d < DT; ++d) vr[d][w] &= keep;
                }
            }
            float c[QT], top[QT];
            bool up = vs.inv > inv_top;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                top[qt] = s[qt][0][0];
#pragma unroll
                for (int j = 1; j < 16; ++j) top[qt] = fmaxf(top[qt], s[qt][j / 4][j % 4]);
                top[qt] = __builtin_fmaf(top[qt], ks, vs.log2);
                c[qt] = quad_max(top[qt]) - kUp;
                up |= c[qt] > mx[qt] + kSlack;
            }
            if (__any(up)) {
                const bool units = __any(vs.inv > inv_top);
                if (units) inv_top = kInvTop;
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
                    const float m2 = fmaxf(mx[qt], c[qt]);
                    const float fade = m2 == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[qt] - m2);
                    float fade_sum = fade;
                    if (units) {
                        const int e1 = unit_exp(un[qt]);
                        const float n2 = fmaxf(quad_max(top[qt] + __builtin_amdgcn_logf(vs.inv)),
                                               mx[qt] - float(e1) + __builtin_amdgcn_logf(quad_sum(sum[qt])));
                        un[qt] = sum_unit(m2 - n2);
                        if (__any(un[qt] != 1.f)) inv_top = -INFINITY;
                        if (m2 != -INFINITY) fade_sum = __builtin_amdgcn_exp2f(mx[qt] - m2 + float(unit_exp(un[qt]) - e1));
                    }
                    mx[qt] = m2;
                    sum[qt] *= fade_sum;
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
                sum[qt] += add == 0.f ? 0.f : add * (vs.inv * un[qt]);  // (a block no row sees may hold NaN)
                pack_p<NV>(p, pf[qt]);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const u32x4 vf = v_operand<FP8, NV>(here(vr[d][2 * hf]), here(vr[d][2 * hf + 1]));
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                        for (int k = 0; k < NV; ++k) o[qt][d] = mfma_v<NV>(vf, pf[qt][hf][k], o[qt][d]);
                    if (hf && d % 2) __builtin_amdgcn_sched_barrier(0);
                }
            vb = vb2;
        }

        // the four waves' sums, brought to one maximum and added (addresses from the thread's
        // number anew: kept over the loop above they would cost it registers)
        const int tid = int(here(threadIdx.x)), el = tid & 15, eg = (tid >> 4) & 3, ew = tid >> 6;
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            sum[qt] = quad_sum(sum[qt]);
            if (eg == 0) {
                m_lds[ew][16 * qt + el] = mx[qt];
                l_lds[ew][16 * qt + el] = sum[qt];
                g_lds[ew][16 * qt + el] = un[qt];
            }
        }
        __syncthreads();
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float m = m_lds[0][16 * qt + el];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) m = fmaxf(m, m_lds[w][16 * qt + el]);
            const float f = mx[qt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[qt] - m);
#pragma unroll
            for (int d = 0; d < DT; ++d)
                *reinterpret_cast<floatx4*>(&o_lds[ew][el][16 * d + 4 * eg]) = o[qt][d] * f;
            __syncthreads();
            const int per = D / 8;
            for (int e = tid; e < 16 * per; e += 64 * kWaves) {
                const int q = e / per, d = 8 * (e - q * per);
                const int r = r0 + 16 * qt + q;
                if (16 * qt + q >= a.rows || r >= rows) continue;
                float mm = m_lds[0][16 * qt + q];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, m_lds[w][16 * qt + q]);
                float l = 0.f, v[8] = {};
                int ee = 0;
                bool far = false;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) far |= g_lds[w][16 * qt + q] != 1.f;
                if (far) {  // a unit for the four sums
                    float nn = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w)
                        nn = fmaxf(nn, m_lds[w][16 * qt + q] - float(unit_exp(g_lds[w][16 * qt + q])) +
                                           __builtin_amdgcn_logf(l_lds[w][16 * qt + q]));
                    ee = unit_exp(sum_unit(mm - nn));
                }
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    const float mw = m_lds[w][16 * qt + q], lw = l_lds[w][16 * qt + q];
                    l += mw == -INFINITY ? lw : lw * __builtin_amdgcn_exp2f(mw - mm + float(ee - unit_exp(g_lds[w][16 * qt + q])));
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] += o_lds[w][q][d + k];
                }
                const int64_t at = (sq.row0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
                const bool direct = F != kParts && whole;
                const float inv = !direct ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = __builtin_amdgcn_ldexpf(v[k] * inv, ee);
                mm -= float(ee);
                if (direct) {
                    store8<true>(static_cast<T*>(a.out) + at * D + d, v);
                    if (a.lse && d == 0) a.lse[at] = l == 0.f ? -INFINITY : mm * kLn2 + __logf(l);
                } else if (F == kParts && !EVEN) {
                    // the prefix's parts, written by the launch before, joined with the row's own
                    const int64_t every = a.b.tokens * a.q_heads;
                    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + at;
                    const float* po = a.part_o + at * D + d;
                    float top = mm;
#pragma unroll 8
                    for (int p = 0; p < pieces; ++p) top = fmaxf(top, ml[p * every].x);
                    const float f0 = mm == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mm - top);
                    float sum_l = mm == -INFINITY ? l : l * f0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= f0;
#pragma unroll 8
                    for (int p = 0; p < pieces; ++p) {
                        const float2 w = ml[p * every];
                        const float f = w.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(w.x - top);
                        sum_l += w.x == -INFINITY ? w.y : w.y * f;
                        float u[8];
                        load8<true>(po + p * every * D, u);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = __builtin_fmaf(u[k], f, v[k]);
                    }
                    const float r = sum_l == 0.f ? 0.f : 1.f / sum_l;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= r;
                    store8<true>(static_cast<T*>(a.out) + at * D + d, v);
                    if (a.lse && d == 0) a.lse[at] = sum_l == 0.f ? -INFINITY : top * kLn2 + __logf(sum_l);
                } else {
                    const int64_t pt = F == kParts && whole ? (shared ? a.solo_a : a.solo_b) + at
                                                            : (F == kParts ? a.slots : 0) + int64_t(slot) * a.rows + 16 * qt + q;
                    store8<true>(a.part_o + pt * D + d, v);
                    if (d == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * pt) = float2{mm, l};
                }
            }
            __syncthreads();
        }
    }
}

template <typename T, bool FP8, int DP, int QT, Form F>
void launch_rows(const AttendDev& d, hipStream_t s) {
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_of(d.blocks), dim3(64 * kWaves), 0, s, d);
    };
    if (d.items)
        d.D == DP ? launch(attend_rows_kernel<T, FP8, DP, QT, true, true, F>)
                  : launch(attend_rows_kernel<T, FP8, DP, QT, false, true, F>);
    else
        d.D == DP ? launch(attend_rows_kernel<T, FP8, DP, QT, true, false, F>)
                  : launch(attend_rows_kernel<T, FP8, DP, QT, false, false, F>);
}
// Rows of a tile: 16 or (headdim 128 at most, not kParts) 32.
template <typename T, bool FP8, Form F>
hipError_t launch_rows_dim(const AttendDev& d, hipStream_t s) {
    if constexpr (F == kParts) {
        if (d.D <= 64) launch_rows<T, FP8, 64, 1, F>(d, s);
        else if (d.D <= 128) launch_rows<T, FP8, 128, 1, F>(d, s);
        else launch_rows<T, FP8, 256, 1, F>(d, s);
    } else {
        const bool one = d.rows == 16;
        if (d.D <= 64) one ? launch_rows<T, FP8, 64, 1, F>(d, s) : launch_rows<T, FP8, 64, 2, F>(d, s);
        else if (d.D <= 128) one ? launch_rows<T, FP8, 128, 1, F>(d, s) : launch_rows<T, FP8, 128, 2, F>(d, s);
        else launch_rows<T, FP8, 256, 1, F>(d, s);
    }
    return hipGetLastError();
}
template <Form F>
hipError_t launch_rows_form(const AttendDev& d, m3_dtype io, hipStream_t s) {
    const bool fp8 = d.c.format == M3_KV_FP8;
    if (io == M3_BF16) return fp8 ? launch_rows_dim<bf16_t, true, F>(d, s) : launch_rows_dim<bf16_t, false, F>(d, s);
    return fp8 ? launch_rows_dim<float, true, F>(d, s) : launch_rows_dim<float, false, F>(d, s);
}

// The launch of a kernel that joins rows' parts: half a wave (a wave above headdim 128) a
// row, or `team` of them.
struct JoinGrid {
    dim3 grid;
    int team;
};
inline JoinGrid join_grid(const AttendDev& d) {
    const int64_t rows = d.b.tokens * d.q_heads;
    const int crews = d.D <= 128 ? 8 : 4;
    int team = 1;  // rows alone fill the chip from about 4 workgroups a CU
    while (team < crews && rows * team / crews < 1024) team *= 2;
    const int per = crews / team;
    return JoinGrid{grid_of((rows + per - 1) / per), team};
}

}  // namespace
}  // namespace m3
