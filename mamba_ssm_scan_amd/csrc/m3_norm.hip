// m3_norm.hip -- the joint between two blocks (m3_norm.h), forward and backward.
//
//   b = s a(g) N(o; w1),  h = x + b,  y = N(h; w2),  N(v; w) = v r w,  r = 1 / sqrt(mean v^2 + eps)
//
// and at (h, o, g), with n = h r2, u = dy w2, n1 = o r1, m = s a(g):
//   dx = dh + r2 (u - n mean(u n))         dw2 = sum dy n
//   v = dx m                               dw1 = sum v n1,  ds = sum dx a(g) N(o)
//   do = r1 (v w1 - n1 mean(v w1 n1))      dg = dx s a'(g) N(o)
//
// Bound by memory. Up to width 4096 every row is read and written once and held in registers
// in between, 8 entries a thread (16 bytes of bf16), so that a row belongs to 16 .. 512 threads
// and a sum over it takes a butterfly in each wave and one exchange through LDS. The vectors
// stay in registers over a workgroup's rows, and the next row's loads are issued before this
// row's sums. 8192 rows of 2048, all parts: forward with an fp32 stream 45 to 49 us (4.8 to 5.2 TB/s),
// backward in bf16 54 + 4 us for the joining of its sums (5.0 TB/s); 16384 of 4096, fp32 stream: 174
// and 269 + 4 us (5.4 and 5.5 TB/s); one step of 128 rows 3.5 us, a launch's least.
//   Above 4096 a row's loads wait for the row before: the forward pass has 1024 threads a row, the
// backward pass 16 entries a thread, and reads each row up to three times. 8192 rows, all parts,
// bytes of one read: width 8192, bf16 156 and 385 us (4.3 and 2.8 TB/s), fp32 stream 182 and 449, fp32 250
// and 607; width 5120, whose last threads idle, bf16 126 and 298 (3.3 and 2.3).
//   Rows that are not 16-byte aligned go entry by entry: 1999 of 1283, fp32, backward 23 + 4 us at 3.5 TB/s
// (16-byte loads at any alignment took 31 us, as the hardware splits them); through the calls, forward
// and backward, 15 and 30 us, in bf16, whose entries are half as wide, 13 and 31. Worst above 4096: 8192 rows of
// 8191 in bf16 176 us and 2.06 ms.
#include <algorithm>

#include "m3_attn_device.h"
#include "m3_norm_internal.h"

namespace m3 {
namespace {

struct NormDev {
    NormArgs a;
    float inv_width;
};
struct NormBackDev {
    NormBackArgs a;
    float inv_width;
    int64_t blocks;
    bool branch, want_o, sums;
};

// 8 entries of a row of TPR threads as they lie in memory: wide, neighbours; else every TPR-th,
// so that a load of a wave covers neighbours too.
template <bool WIDE, int TPR>
__device__ __forceinline__ int column(int c, int k, int tid) {
    return WIDE ? (c * TPR + tid) * 8 + k : (c * 8 + k) * TPR + tid;
}
template <typename T, bool WIDE>
struct Raw;
template <>
struct Raw<bf16_t, true> {
    u32x4 w;
};
template <>
struct Raw<float, true> {
    floatx4 w[2];
};
template <typename T>
struct Raw<T, false> {
    T w[8];
};
template <typename T, bool WIDE, int TPR>
__device__ __forceinline__ void fetch(Raw<T, WIDE>& r, const T* row, int c, int tid, int width, bool live) {
    if constexpr (WIDE) {
        const int at = column<true, TPR>(c, 0, tid);
        r = {};
        if (live && at < width) r = *reinterpret_cast<const Raw<T, WIDE>*>(row + at);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int at = column<false, TPR>(c, k, tid);
            r.w[k] = T{};
            if (live && at < width) r.w[k] = row[at];
        }
    }
}
__device__ __forceinline__ void values(const Raw<bf16_t, true>& r, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(r.w[j] << 16);
        v[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void values(const Raw<float, true>& r, float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r.w[j / 4][j % 4];
}
__device__ __forceinline__ void values(const Raw<bf16_t, false>& r, float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = bf16_to_f32(r.w[j].bits);
}
__device__ __forceinline__ void values(const Raw<float, false>& r, float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r.w[j];
}
template <typename T, bool WIDE, int TPR>
__device__ __forceinline__ void put(T* row, int c, int tid, int width, const float* v) {
    if constexpr (WIDE) {
        const int at = column<true, TPR>(c, 0, tid);
        if (at < width) store8<true>(row + at, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int at = column<false, TPR>(c, k, tid);
            if (at < width) Io<T>::store(row, at, v[k]);
        }
    }
}
// 8 entries of a vector, times f (all f where there is none)
template <bool WIDE, int TPR>
__device__ __forceinline__ void vector8(const float* p, float f, int c, int tid, int width, float* v) {
    if (p) {
        Raw<float, WIDE> r;
        fetch<float, WIDE, TPR>(r, p, c, tid, width, true);
        values(r, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= f;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = f;
    }
}

// Squares are summed as 2^-6 of themselves, an exact scaling: a full row of 8192 entries of
// 2^60 stays in range (2^127).
constexpr float kSquare = 0x1p-6f;
__device__ __forceinline__ float add_square(float v, float s) { return __builtin_fmaf(v * kSquare, v, s); }
// 1 / sqrt(mean v^2 + eps) of such a sum
__device__ __forceinline__ float inverse_rms(float s, float inv_width, float eps) {
    return __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_width * (1.f / kSquare), eps));
}

// Sums over a row's threads, the same bits in each. More than a wave: through LDS, two
// buffers in turn, so that one barrier a sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*lds)[1024 / 64][3], int& turn) {
#pragma unroll
    for (int k = 1; k < (TPR < 64 ? TPR : 64); k <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) s[n] += __shfl_xor(s[n], k);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x / 64, first = wave / (TPR / 64) * (TPR / 64);
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) lds[turn][wave][n] = s[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            s[n] = 0.f;
#pragma unroll
            for (int w = 0; w < TPR / 64; ++w) s[n] += lds[turn][first + w][n];
        }
        turn ^= 1;
    }
}

// a(g) and its slope
__device__ __forceinline__ float gate_of(int fn, float g) {
    return fn == M3_GATE_IDENTITY ? g : fn == M3_GATE_SILU ? g * sigmoid_f(g) : sigmoid_f(g);
}
__device__ __forceinline__ void gate_of(int fn, float g, float* act, float* slope) {
    if (fn == M3_GATE_IDENTITY) {
        *act = g;
        *slope = 1.f;
        return;
    }
    const float s = sigmoid_f(g), rest = sigmoid_f(-g);  // (1 - s would lose a small rest)
    *act = fn == M3_GATE_SILU ? g * s : s;
    *slope = fn == M3_GATE_SILU ? s * __builtin_fmaf(g, rest, 1.f) : s * rest;
}

// the launch's workgroup: TPR threads a row, 256 at least
template <int TPR>
constexpr int kForwardThreads = TPR < 256 ? 256 : TPR;

template <typename X, typename T, int TPR, int CH, bool WIDE>
__global__ __launch_bounds__(kForwardThreads<TPR>) void joint_kernel(NormDev d) {
    constexpr int NT = kForwardThreads<TPR>, RPW = NT / TPR;
    constexpr bool kAhead = TPR <= 512;  // (above width 4096 a row is loaded after the one before)
    __shared__ float lds[2][1024 / 64][3];
    const NormArgs& a = d.a;
    const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR, width = a.j.width;
    const bool branch = a.o.p, gated = a.gate.p;
    int turn = 0;
    float w1[CH][8], w2[CH][8], sc[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        vector8<WIDE, TPR>(a.j.post_weight, 1.f, c, tid, width, w1[c]);
        vector8<WIDE, TPR>(a.j.weight, 1.f, c, tid, width, w2[c]);
        vector8<WIDE, TPR>(a.j.scale, a.j.factor, c, tid, width, sc[c]);
    }
    struct Row {
        Raw<X, WIDE> x[CH];
        Raw<T, WIDE> o[CH], g[CH];
    };
    auto load = [&](Row& r, int64_t row) {
        const bool live = row < a.j.tokens;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            fetch<X, WIDE, TPR>(r.x[c], static_cast<const X*>(a.x.p) + row * a.x.stride, c, tid, width, live);
            fetch<T, WIDE, TPR>(r.o[c], static_cast<const T*>(a.o.p) + row * a.o.stride, c, tid, width, live && branch);
            fetch<T, WIDE, TPR>(r.g[c], static_cast<const T*>(a.gate.p) + row * a.gate.stride, c, tid, width, live && gated);
        }
    };
    const int64_t step = int64_t(gridDim.x) * RPW;
    int64_t row0 = int64_t(blockIdx.x) * RPW;
    Row now, next;
    load(now, row0 + sub);
    for (; row0 < a.j.tokens; row0 += step) {
        const int64_t row = row0 + sub;
        if constexpr (kAhead) load(next, row + step);
        float h[CH][8];
#pragma unroll
        for (int c = 0; c < CH; ++c) values(now.x[c], h[c]);
        if (branch) {
            float r1 = 1.f;
            if (a.j.post_weight) {
                float s[1] = {0.f};
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float o[8];
                    values(now.o[c], o);
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[0] = add_square(o[k], s[0]);
                }
                row_sum<TPR, 1>(s, lds, turn);
                r1 = inverse_rms(s[0], d.inv_width, a.j.eps);
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float o[8], g[8];
                values(now.o[c], o);
                values(now.g[c], g);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float act = gated ? gate_of(a.j.gate_fn, g[k]) : 1.f;
                    h[c][k] = __builtin_fmaf(o[k] * r1 * w1[c][k] * act, sc[c][k], h[c][k]);
                }
            }
            if (row < a.j.tokens) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    put<X, WIDE, TPR>(static_cast<X*>(a.h.p) + row * a.h.stride, c, tid, width, h[c]);
            }
        }
        if (a.j.weight) {
            float s[1] = {0.f};
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k) s[0] = add_square(h[c][k], s[0]);
            row_sum<TPR, 1>(s, lds, turn);
            const float r2 = inverse_rms(s[0], d.inv_width, a.j.eps);
            if (row < a.j.tokens) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[c][k] *= r2 * w2[c][k];
                    put<T, WIDE, TPR>(static_cast<T*>(a.y.p) + row * a.y.stride, c, tid, width, h[c]);
                }
            }
        }
        if constexpr (kAhead) now = next;
        else load(now, row + step);
    }
}

// In the last column block of a row beyond `width` the raw entries are 0, so that no sum
// takes anything from there; what is formed there is not stored.
template <typename X, typename T, int TPR, int CH, bool WIDE>
__global__ __launch_bounds__(kNormBackThreads) void joint_back_kernel(NormBackDev d) {
    constexpr int NT = kNormBackThreads, RPW = NT / TPR;
    // above 4096 entries nothing of a row is kept: it is read again (from L2) for each phase
    constexpr bool kHold = CH == 1;
    __shared__ float lds[2][1024 / 64][3];
    __shared__ float fold[RPW > 1 ? NT * 8 : 1];
    const NormBackArgs& a = d.a;
    int tid = threadIdx.x % TPR;
    const int sub = threadIdx.x / TPR, width = a.j.width;
    const bool normed = a.j.weight, branch = d.branch, post = branch && a.j.post_weight, gated = branch && a.gate.p;
    int turn = 0;
    float acc[3][CH][8];
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[q][c][k] = 0.f;
    float hw1[8], hw2[8], hsc[8];
    auto vectors = [&](int c) {
        vector8<WIDE, TPR>(a.j.post_weight, 1.f, c, tid, width, hw1);
        vector8<WIDE, TPR>(a.j.weight, 1.f, c, tid, width, hw2);
        vector8<WIDE, TPR>(a.j.scale, a.j.factor, c, tid, width, hsc);
    };
    if constexpr (kHold) vectors(0);
    struct Row {
        Raw<X, WIDE> dh, h;
        Raw<T, WIDE> dy, o, g;
    };
    auto load = [&](Row& r, int64_t row, int c) {
        const bool live = row < a.j.tokens;
        fetch<X, WIDE, TPR>(r.h, static_cast<const X*>(a.h.p) + row * a.h.stride, c, tid, width, live && normed);
        fetch<X, WIDE, TPR>(r.dh, static_cast<const X*>(a.dh.p) + row * a.dh.stride, c, tid, width, live && a.dh.p);
        fetch<T, WIDE, TPR>(r.dy, static_cast<const T*>(a.dy.p) + row * a.dy.stride, c, tid, width, live && normed);
        fetch<T, WIDE, TPR>(r.o, static_cast<const T*>(a.o.p) + row * a.o.stride, c, tid, width, live && branch);
        fetch<T, WIDE, TPR>(r.g, static_cast<const T*>(a.gate.p) + row * a.gate.stride, c, tid, width, live && gated);
    };
    const int64_t step = int64_t(gridDim.x) * RPW;
    int64_t row0 = int64_t(blockIdx.x) * RPW;
    Row now, next;
    if constexpr (kHold) load(now, row0 + sub, 0);
    for (; row0 < a.j.tokens; row0 += step) {
        const int64_t row = row0 + sub;
        if constexpr (kHold) load(next, row + step, 0);
        auto bring = [&](int c) {
            if constexpr (!kHold) {
                // one piece at a time, read and addressed anew: else all of them take registers
                asm volatile("" : "+v"(tid)::"memory");
                __builtin_amdgcn_sched_barrier(0);
                load(now, row, c);
                vectors(c);
            }
        };
        float r2 = 0.f, back = 0.f, r1 = 1.f;  // back: r2^2 mean(u h) of the norm of h
        if (normed || post) {
            float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                bring(c);
                float h[8], dy[8], o[8];
                values(now.h, h);
                values(now.dy, dy);
                values(now.o, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s[0] = add_square(h[k], s[0]);
                    s[1] = __builtin_fmaf(dy[k] * hw2[k], h[k], s[1]);
                    s[2] = add_square(o[k], s[2]);
                }
            }
            row_sum<TPR, 3>(s, lds, turn);
            r2 = normed ? inverse_rms(s[0], d.inv_width, a.j.eps) : 0.f;
            back = s[1] * r2 * d.inv_width * r2;
            if (post) r1 = inverse_rms(s[2], d.inv_width, a.j.eps);
        }
        // the stream's gradient, and the branch's parts: act, slope, v
        float t[8], act[8], slope[8], n1[8];
        auto parts = [&]() {
            float h[8], dy[8], o[8], g[8];
            values(now.dh, t);
            values(now.h, h);
            values(now.dy, dy);
            values(now.o, o);
            values(now.g, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (normed) t[k] = __builtin_fmaf(r2, __builtin_fmaf(-h[k], back, dy[k] * hw2[k]), t[k]);
                act[k] = slope[k] = 1.f;
                if (gated) gate_of(a.j.gate_fn, g[k], &act[k], &slope[k]);
                n1[k] = o[k] * r1;
            }
        };
        float mean = 0.f;  // mean(v w1 n1)
        if (post && d.want_o) {
            float s[1] = {0.f};
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                bring(c);
                parts();
#pragma unroll
                for (int k = 0; k < 8; ++k) s[0] = __builtin_fmaf(t[k] * act[k] * hsc[k] * hw1[k], n1[k], s[0]);
            }
            row_sum<TPR, 1>(s, lds, turn);
            mean = s[0] * d.inv_width;
        }
        if (row < a.j.tokens) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                bring(c);
                if (!(kHold && post && d.want_o)) parts();
                float h[8], dy[8], out[8];
                if (a.dx.p) put<X, WIDE, TPR>(static_cast<X*>(a.dx.p) + row * a.dx.stride, c, tid, width, t);
                if (d.sums && normed) {
                    values(now.h, h);
                    values(now.dy, dy);
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[0][c][k] = __builtin_fmaf(dy[k] * r2, h[k], acc[0][c][k]);
                }
                if (!branch) continue;
                if (a.d_gate.p) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) out[k] = t[k] * hsc[k] * slope[k] * n1[k] * hw1[k];
                    put<T, WIDE, TPR>(static_cast<T*>(a.d_gate.p) + row * a.d_gate.stride, c, tid, width, out);
                }
                if (d.sums) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float x = t[k] * act[k] * n1[k];
                        acc[1][c][k] = __builtin_fmaf(x, hsc[k], acc[1][c][k]);
                        acc[2][c][k] = __builtin_fmaf(x, hw1[k], acc[2][c][k]);
                    }
                }
                if (a.d_o.p) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float v = t[k] * act[k] * hsc[k];
                        out[k] = post ? r1 * __builtin_fmaf(-n1[k], mean, v * hw1[k]) : v;
                    }
                    put<T, WIDE, TPR>(static_cast<T*>(a.d_o.p) + row * a.d_o.stride, c, tid, width, out);
                }
            }
        }
        if constexpr (kHold) now = next;
    }
    if (!d.sums) return;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        if (!a.sums[q]) continue;
        float* part = a.parts + (q * d.blocks + blockIdx.x) * width;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = q == 2 ? acc[q][c][k] * a.j.factor : acc[q][c][k];
            if constexpr (RPW > 1) {  // the workgroup's rows side by side, added in their order
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 8; ++k) fold[k * NT + threadIdx.x] = v[k];
                __syncthreads();
                if (sub) continue;
                for (int s = 1; s < RPW; ++s)
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] += fold[k * NT + s * TPR + tid];
            }
            put<float, WIDE, TPR>(part, c, tid, width, v);
        }
    }
}

// The workgroups' parts of a sum added up: 64 columns a workgroup, every 8th part a wave.
__global__ __launch_bounds__(512) void joint_sums_kernel(NormBackDev d) {
    __shared__ float lds[8][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, at = blockIdx.x * 64 + lane, q = blockIdx.y;
    const int width = d.a.j.width;
    float* out = d.a.sums[q];
    if (!out) return;
    float s = 0.f;
    if (at < width) {
        const float* p = d.a.parts + q * d.blocks * width + at;
#pragma unroll 8
        for (int64_t b = wave; b < d.blocks; b += 8) s += p[b * width];
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave || at >= width) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) s += lds[w][lane];
    out[at] = s;
}

// f(threads of a row, pieces of 8 a thread) as compile-time numbers
template <int N>
struct Int {
    static constexpr int v = N;
};
template <int MOST, typename F>
void with_row(int width, bool wide, F f) {
    switch (norm_row_threads(width, wide, MOST)) {
        case 16: return f(Int<16>{}, Int<1>{});
        case 64: return f(Int<64>{}, Int<1>{});
        case 128: return f(Int<128>{}, Int<1>{});
        case 256: return f(Int<256>{}, Int<1>{});
    }
    if (width <= 4096) return f(Int<512>{}, Int<1>{});
    f(Int<MOST>{}, Int<kNormWidth / (8 * MOST)>{});
}
// g(stream type, io type, wide)
template <int TPR, typename G>
void with_types(const m3_joint& j, bool wide, G g) {
    auto types = [&](auto w) {
        if (j.stream_dtype == M3_BF16) g(bf16_t{}, bf16_t{}, w);
        else if (j.io_dtype == M3_BF16) g(float{}, bf16_t{}, w);
        else g(float{}, float{}, w);
    };
    if (wide) return types(Int<1>{});
    if constexpr (TPR >= 64) types(Int<0>{});
}

}  // namespace

hipError_t launch_norm(const NormArgs& a) {
    const NormDev d{a, 1.f / float(a.j.width)};
    with_row<kNormForwardMost>(a.j.width, a.wide, [&](auto tpr, auto ch) {
        constexpr int TPR = decltype(tpr)::v, CH = decltype(ch)::v, NT = kForwardThreads<TPR>;
        const int64_t groups = (a.j.tokens + NT / TPR - 1) / (NT / TPR);
        const unsigned grid = unsigned(std::min<int64_t>(groups, 256 * 1024 / NT));
        with_types<TPR>(a.j, a.wide, [&](auto x, auto t, auto w) {
            hipLaunchKernelGGL((joint_kernel<decltype(x), decltype(t), TPR, CH, decltype(w)::v != 0>), dim3(grid), dim3(NT), 0,
                               a.stream, d);
        });
    });
    return hipGetLastError();
}

hipError_t launch_norm_back(const NormBackArgs& a) {
    const int width = a.j.width;
    const bool sums = a.sums[0] || a.sums[1] || a.sums[2];
    const bool branch = a.d_o.p || a.d_gate.p || a.sums[1] || a.sums[2];
    const NormBackDev d{a, 1.f / float(width), norm_back_blocks(a.j.tokens, width, a.wide), branch, a.d_o.p != nullptr, sums};
    if (d.blocks > 0)
        with_row<kNormBackThreads>(width, a.wide, [&](auto tpr, auto ch) {
            constexpr int TPR = decltype(tpr)::v, CH = decltype(ch)::v;
            with_types<TPR>(a.j, a.wide, [&](auto x, auto t, auto w) {
                hipLaunchKernelGGL((joint_back_kernel<decltype(x), decltype(t), TPR, CH, decltype(w)::v != 0>),
                                   dim3(unsigned(d.blocks)), dim3(kNormBackThreads), 0, a.stream, d);
            });
        });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !sums) return e;
    hipLaunchKernelGGL(joint_sums_kernel, dim3(unsigned((width + 63) / 64), 3), dim3(512), 0, a.stream, d);
    return hipGetLastError();
}

}  // namespace m3
