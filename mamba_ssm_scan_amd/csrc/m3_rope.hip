// m3_rope.hip -- rotary positions on rows of heads, and their transposed map
// (the gradient).
//
// y = R(theta) x per pair: 6 flops for 2 entries read and written, so the copy
// rate is the floor. A workgroup takes a few tokens: its threads first form
// the tokens' (cos, sin) once, in fp64, into LDS, then walk the tokens' heads
// in pieces of 8 entries held in registers (half layout: the piece and its
// partner rot / 2 further on), so the angles' cost is shared by all heads and
// every entry is read and written once, 16 bytes a lane. 8192 tokens of 32 heads of 64
// (bf16): 11.9 us, 5.6 TB/s of reads and writes; 128 tokens of 16 heads of 128: 3.0 us,
// a launch.
#include "m3_attn_device.h"
#include "m3_attn_internal.h"

namespace m3 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 1024;  // (cos, sin) pairs of the tokens of a workgroup held in LDS

struct RopeDev {
    const void* x;
    void* y;
    const int32_t* positions;
    const float* inv_freq;
    int64_t x_tok, x_head, y_tok, y_head, tokens;
    int heads, D, half;  // half = rot / 2
    int tb;              // tokens of a workgroup
    float mscale;
    float sign;          // -1: the transposed map
    int interleaved;
};

__device__ __forceinline__ void angles(const RopeDev& a, int64_t t0, int nt, float2* cs) {
    for (int e = threadIdx.x; e < nt * a.half; e += kThreads) {
        const int t = e / a.half, i = e - t * a.half;
        float c, s;
        cos_sin(a.positions[t0 + t], a.inv_freq[i], double(a.mscale), &c, &s);
        cs[e] = float2{c, a.sign * s};
    }
    __syncthreads();
}

// Pieces of 8 entries. Half layout (rot a multiple of 16): piece j < rot / 16
// and piece j + rot / 16 turn together; interleaved (rot a multiple of 8): each
// piece holds 4 pairs. The pieces after rot are copied.
template <typename T, bool INTER>
__global__ __launch_bounds__(kThreads) void rope_wide_kernel(RopeDev a) {
    __shared__ float2 cs[kMaxPairs];
    const int64_t t0 = int64_t(block_id()) * a.tb;
    if (t0 >= a.tokens) return;
    const int nt = int(min(int64_t(a.tb), a.tokens - t0));
    angles(a, t0, nt, cs);
    const int turned = INTER ? a.half / 4 : a.half / 8;          // pieces (pairs of pieces) that turn
    const int per = turned + (a.D - 2 * a.half) / 8;             // jobs of a head
    const int jobs = a.heads * per;
    for (int e = threadIdx.x; e < nt * jobs; e += kThreads) {
        const int t = e / jobs, r = e - t * jobs, h = r / per, j = r - h * per;
        const T* x = static_cast<const T*>(a.x) + (t0 + t) * a.x_tok + h * a.x_head;
        T* y = static_cast<T*>(a.y) + (t0 + t) * a.y_tok + h * a.y_head;
        float u[8], v[8];
        if (j >= turned) {
            const int d = 2 * a.half + 8 * (j - turned);
            load8<true>(x + d, u);
            store8<true>(y + d, u);
        } else if constexpr (INTER) {
            load8<true>(x + 8 * j, u);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2 w = cs[t * a.half + 4 * j + p];
                turn(u[2 * p], u[2 * p + 1], w.x, w.y);
            }
            store8<true>(y + 8 * j, u);
        } else {
            load8<true>(x + 8 * j, u);
            load8<true>(x + a.half + 8 * j, v);
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float2 w = cs[t * a.half + 8 * j + p];
                turn(u[p], v[p], w.x, w.y);
            }
            store8<true>(y + 8 * j, u);
            store8<true>(y + a.half + 8 * j, v);
        }
    }
}

// Any size, stride and alignment: one pair, or one copied entry, per thread and
// step. rot / 2 above kMaxPairs forms the angles where they are used.
template <typename T>
__global__ __launch_bounds__(kThreads) void rope_any_kernel(RopeDev a) {
    __shared__ float2 cs[kMaxPairs];
    const int64_t t0 = int64_t(block_id()) * a.tb;
    if (t0 >= a.tokens) return;
    const int nt = int(min(int64_t(a.tb), a.tokens - t0));
    const bool held = a.half <= kMaxPairs;
    if (held) angles(a, t0, nt, cs);
    const int per = a.half + (a.D - 2 * a.half);
    const int64_t jobs = int64_t(a.heads) * per;
    for (int64_t e = threadIdx.x; e < nt * jobs; e += kThreads) {
        const int64_t t = e / jobs, r = e - t * jobs;
        const int h = int(r / per), j = int(r - int64_t(h) * per);
        const T* x = static_cast<const T*>(a.x) + (t0 + t) * a.x_tok + h * a.x_head;
        T* y = static_cast<T*>(a.y) + (t0 + t) * a.y_tok + h * a.y_head;
        if (j >= a.half) {
            Io<T>::store(y, a.half + j, Io<T>::load(x, a.half + j));
            continue;
        }
        float2 w;
        if (held) {
            w = cs[t * a.half + j];
        } else {
            float c, s;
            cos_sin(a.positions[t0 + t], a.inv_freq[j], double(a.mscale), &c, &s);
            w = float2{c, a.sign * s};
        }
        const int i0 = a.interleaved ? 2 * j : j, i1 = a.interleaved ? 2 * j + 1 : j + a.half;
        float u = Io<T>::load(x, i0), v = Io<T>::load(x, i1);
        turn(u, v, w.x, w.y);
        Io<T>::store(y, i0, u);
        Io<T>::store(y, i1, v);
    }
}

template <typename T>
hipError_t launch(const RopeArgs& a) {
    RopeDev d{a.x, a.y, a.positions, a.rot.inv_freq, a.x_tok, a.x_head, a.y_tok, a.y_head, a.tokens,
              a.heads, a.D, a.rot.rot / 2, 1, a.rot.mscale, a.backward ? -1.f : 1.f, a.rot.interleaved};
    // tokens of a workgroup: enough work for its threads (2 pieces of 16 entries
    // each), as many angles as LDS holds, and no fewer workgroups than 4 per CU
    const int64_t entries = int64_t(a.heads) * a.D;
    int64_t tb = std::min<int64_t>((2 * kThreads * 16 + entries - 1) / entries, std::max(1, kMaxPairs / d.half));
    tb = std::max<int64_t>(1, std::min<int64_t>(tb, a.tokens / 1024));
    d.tb = int(tb);
    const dim3 grid = grid_of((a.tokens + tb - 1) / tb);
    const bool inter = a.rot.interleaved != 0;
    if (a.wide && a.D % 8 == 0 && a.rot.rot % (inter ? 8 : 16) == 0 && d.half <= kMaxPairs) {
        if (inter)
            hipLaunchKernelGGL((rope_wide_kernel<T, true>), grid, dim3(kThreads), 0, a.stream, d);
        else
            hipLaunchKernelGGL((rope_wide_kernel<T, false>), grid, dim3(kThreads), 0, a.stream, d);
    } else {
        hipLaunchKernelGGL((rope_any_kernel<T>), grid, dim3(kThreads), 0, a.stream, d);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a) {
    return a.io == M3_BF16 ? launch<bf16_t>(a) : launch<float>(a);
}

}  // namespace m3
