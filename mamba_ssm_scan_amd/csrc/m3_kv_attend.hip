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
// waves): 8.5 and 4.5 us. 16 sequences of 8000 with 4 rows each (16 heads over 4 of 128): 36
// us, of 64 of 2000 in fp32 (8 over 2) 29.
#include <algorithm>

#include "m3_attend_common.h"

namespace m3 {
namespace {

constexpr int kWaves = 4;
constexpr int kMaxItems = kAttendItems;

// Even shares. The tiles of all (sequence, row tile) items lie one after the other,
// an item's once for each key head; a workgroup takes the same number of them,
// whatever the lengths, and a row tile's keys that several share are joined
// afterwards. An item's keys for one head are one run: the share that holds its
// first tile but not its last writes part 0 to its slot 2 w + 1, a later share w
// the next part to slot 2 w. Every workgroup forms the items' first tiles itself
// (one scan of the lengths), the first also stores them for the join. Returns the
// tiles of a share: a multiple of 4, one tile a wave at least.
template <bool VIEW>
__device__ __forceinline__ int even_shares(const AttendDev& a, int* first, int* scan) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (a.items + 64 * kWaves - 1) / (64 * kWaves);
    const int e0 = threadIdx.x * per, e1 = min(e0 + per, a.items);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        const Unit u = pair_of(a, e);
        const Seq sq = seq_of(a.b, u.i);
        const int64_t r0 = u.at * a.rows;
        const Span sp = r0 >= 0 && r0 < sq.n * a.group ? span_of<VIEW>(a, sq, int(r0)) : Span{0, 0, 0, 0};
        first[e] = int(sp.hi - sp.lo);
        sum += int(sp.hi - sp.lo);
    }
    int up = sum;  // over the wave, then over the waves before
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const int o = __shfl_up(up, k);
        up += lane >= k ? o : 0;
    }
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
    const int share = int((all + 4 * a.blocks - 1) / (4 * a.blocks)) * 4;
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
// Waves a SIMD: what the registers of each case allow without spilling in its loop.
template <typename T, int DP, int QT, bool EVEN, bool VIEW>
constexpr int kSimdWaves = DP == 256 || (sizeof(T) == 4 && DP * QT > 128) || (VIEW && EVEN && DP * QT > 128) ? 1
                           : sizeof(T) == 4 || QT == 2                                                        ? 2
                           : DP == 64                                                                         ? 4
                           : EVEN || VIEW                                                                     ? 2
                                                                                                              : 3;
template <typename T, bool FP8, int DP, int QT, bool FULL, bool EVEN, bool VIEW>
__global__ __launch_bounds__(64 * kWaves, (kSimdWaves<T, DP, QT, EVEN, VIEW>)) void attend_rows_kernel(AttendDev a) {
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
    __shared__ int scan_lds[kWaves];
    const int w = int(block_id());
    if (w >= a.blocks) return;
    int64_t x = 0, xe = 1;  // what is left of this workgroup's share
    if constexpr (EVEN) {
        const int share = even_shares<VIEW>(a, first_lds, scan_lds);
        x = int64_t(w) * share;
        xe = min(x + share, int64_t(H) * first_lds[a.items]);
        zero_rows<T>(a, first_lds);
    }
    while (x < xe) {  // (a share may end one row tile's keys and begin the next's)
        int64_t i, rt;
        int h, t0 = 0, t1 = 0;
        bool whole = true;
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
            const Unit u = pair_of(a, e);
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
        const Seq sq = seq_of(a.b, i);
        const int rows = sq.n * a.group;
        if (rt < 0 || rt * a.rows >= rows) break;  // (without shares only)
        const int r0 = int(rt) * a.rows;
        const int64_t base = sq.base;
        const Span sp = span_of<VIEW>(a, sq, r0);
        const int slot = t0 > 0 ? 2 * w : 2 * w + 1;
        if constexpr (EVEN) {
            t0 += int(sp.lo);
            t1 += int(sp.lo);
        } else {
            t0 = int(sp.lo);
            t1 = int(sp.hi);
        }
        if (a.c.num_pages == 0) t1 = t0;

        const int D = FULL ? DP : a.D;
        const int held = int(min(int64_t(sq.held), a.b.max_kv)), held_blocks = (held + 15) / 16;
        const int32_t* pages = a.b.pages + i * a.b.max_pages;
        // (VIEW) keys that sinks show, the first block that the window does, and the shared pages
        const int sinks = VIEW ? int(a.view.sinks) : 0, sink_blocks = (sinks + 15) / 16;
        const int win_block = VIEW && a.window ? int(max(base + r0 / a.group - a.window + 1, int64_t(0)) / 16) : 0;
        const Prefix pre = VIEW ? prefix_of(a, i) : Prefix{nullptr, 0};
        auto find = [&](int blk) {  // a block's index for this head, -1: none (there are fewer than 2^31)
            const int pg = blk >> a.shift;
            if (blk >= held_blocks || (!VIEW && pg >= a.b.max_pages)) return -1;  // (max_kv ends in the table)
            if (VIEW && blk < win_block && blk >= sink_blocks) return -1;
            const int64_t p = VIEW && pg < pre.count ? pre.pages[pg] : pages[pg];
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
            const int at = tile_at<VIEW>(sp, tile);
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
            khi[qt] = !live ? 0 : a.causal ? int(min(int64_t(held), base + tok + 1)) : held;
            klo[qt] = !live || !a.window ? 0 : int(max(base + tok - a.window + 1, int64_t(0)));
        }
        // keys that every row sees: tiles inside need no mask
        const int rl = min(r0 + a.rows, rows) - 1;
        const int all_hi = a.causal ? int(max(min(int64_t(held), base + r0 / a.group + 1), int64_t(0))) : held;
        const int all_lo = a.window ? int(max(base + rl / a.group - a.window + 1, int64_t(0))) : 0;

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
            const int k0 = tile_at<VIEW>(sp, tile) * kTile, next = tile + kWaves;
            int kb2 = -1, vb2 = -1;
            if (next < t1) {
                const int at = tile_at<VIEW>(sp, next);
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
            if ((k0 < all_lo && (!VIEW || k0 + kTile > sinks)) || k0 + kTile > all_hi || __any(!there || !(ks >= 0.f) || vs.none)) {
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int key = k0 + 16 * g + j;
                        const float x = __builtin_fmaf(s[qt][j / 4][j % 4], ks, vs.log2);
                        s[qt][j / 4][j % 4] = there && (key >= klo[qt] || (VIEW && key < sinks)) && key < khi[qt] ? x : -INFINITY;
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
                const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = __builtin_amdgcn_ldexpf(v[k] * inv, ee);
                mm -= float(ee);
                if (whole) {
                    store8<true>(static_cast<T*>(a.out) + at * D + d, v);
                    if (a.lse && d == 0) a.lse[at] = l == 0.f ? -INFINITY : mm * kLn2 + __logf(l);
                } else {
                    const int64_t pt = int64_t(slot) * a.rows + 16 * qt + q;
                    store8<true>(a.part_o + pt * D + d, v);
                    if (d == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * pt) = float2{mm, l};
                }
            }
            __syncthreads();
        }
    }
}

// Joins rows' parts, in their order. Half a wave (a wave above headdim 128) takes a
// row's parts, or `team` of them do where there are few rows (team: a power of two).
template <typename T, bool VIEW>
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
        const Span sp = live ? span_of<VIEW>(a, sq, r / a.rows * a.rows) : Span{0, 0, 0, 0};
        parts = cut_of(a, sp).pieces;
        live = live && parts > 1;
        p0 = p1 = at;
        step = a.b.tokens * a.q_heads;
    }
    if (!live) parts = 0;
    auto place = [&](int p) { return p ? p1 + p * step : p0; };
    float m = -INFINITY;
    for (int p = lane; p < parts; p += width) m = fmaxf(m, a.part_ml[2 * place(p)]);
    for (int x = 1; x < width; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    float l = 0.f;
    for (int p = lane; p < parts; p += width) {
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * place(p));
        l += ml.x == -INFINITY ? ml.y : ml.y * __builtin_amdgcn_exp2f(ml.x - m);
    }
    for (int x = 1; x < width; x <<= 1) l += __shfl_xor(l, x);
    floatx4 v{0, 0, 0, 0};
    if (4 * lane < D) {
#pragma unroll 4
        for (int p = member; p < parts; p += team) {
            const float mp = a.part_ml[2 * place(p)];
            const float f = mp == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mp - m);
            v += *reinterpret_cast<const floatx4*>(a.part_o + place(p) * D + 4 * lane) * f;
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
hipError_t launch_join(const AttendDev& d, hipStream_t s) {
    const int64_t rows = d.b.tokens * d.q_heads;
    const int crews = d.D <= 128 ? 8 : 4;
    int team = 1;  // rows alone fill the chip from about 4 workgroups a CU
    while (team < crews && rows * team / crews < 1024) team *= 2;
    const int per = crews / team;
    const dim3 grid = grid_of((rows + per - 1) / per);
    if (has_view(d.view)) hipLaunchKernelGGL((attend_join_kernel<T, true>), grid, dim3(256), 0, s, d, team);
    else hipLaunchKernelGGL((attend_join_kernel<T, false>), grid, dim3(256), 0, s, d, team);
    return hipGetLastError();
}

template <typename T, bool FP8, int DP, int QT, bool VIEW>
void launch_rows_of(const AttendDev& d, hipStream_t s) {
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_of(d.blocks), dim3(64 * kWaves), 0, s, d);
    };
    if (d.items)
        d.D == DP ? launch(attend_rows_kernel<T, FP8, DP, QT, true, true, VIEW>)
                  : launch(attend_rows_kernel<T, FP8, DP, QT, false, true, VIEW>);
    else
        d.D == DP ? launch(attend_rows_kernel<T, FP8, DP, QT, true, false, VIEW>)
                  : launch(attend_rows_kernel<T, FP8, DP, QT, false, false, VIEW>);
}
template <typename T, bool FP8, int DP, int QT>
void launch_rows(const AttendDev& d, hipStream_t s) {
    has_view(d.view) ? launch_rows_of<T, FP8, DP, QT, true>(d, s) : launch_rows_of<T, FP8, DP, QT, false>(d, s);
}
template <typename T, bool FP8>
hipError_t launch_attend(const AttendArgs& a) {
    const AttendPlan& p = a.plan;
    char* ws = static_cast<char*>(a.workspace);
    AttendDev d{a.c, a.b, a.q, a.out, a.lse, reinterpret_cast<float*>(ws + p.o_off),
                reinterpret_cast<float*>(ws + p.ml_off), reinterpret_cast<int*>(ws), p.items,
                p.packed ? __builtin_ctz(unsigned(p.rows)) : 0, a.q_heads,
                a.q_heads / a.c.heads, a.c.headdim, __builtin_ctz(unsigned(a.c.page_size / 16)), p.rows,
                a.scale * kLog2e, a.view.causal, a.view.window, p.row_tiles, p.split_tiles, p.splits, a.wide, p.blocks, a.view,
                0, 0};
    if (p.tile) {
        const hipError_t e = launch_attend_tile(d, a.io, a.stream);
        return e != hipSuccess || p.splits == 1 ? e : launch_join<T>(d, a.stream);
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
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || !p.items ? e : launch_join<T>(d, a.stream);
}

}  // namespace

hipError_t launch_kv_attend(const AttendArgs& a) {
    const bool fp8 = a.c.format == M3_KV_FP8;
    if (a.io == M3_BF16) return fp8 ? launch_attend<bf16_t, true>(a) : launch_attend<bf16_t, false>(a);
    return fp8 ? launch_attend<float, true>(a) : launch_attend<float, false>(a);
}

}  // namespace m3
