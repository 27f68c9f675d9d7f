// m3_norm_internal.h -- what the joint's entry points (m3_norm_host.cpp) hand to
// its kernel launchers (m3_norm.hip). Not part of the public ABI.
#pragma once
#include "../../include/m3_norm.h"
#include "m3_internal.h"

namespace m3 {

// Absent rows have p NULL.
struct NormArgs {
    m3_joint j;
    m3_lines x, o, gate, h, y;
    bool wide;  // pointers, strides and the width take 16-byte accesses
    hipStream_t stream;
};
hipError_t launch_norm(const NormArgs& a);

struct NormBackArgs {
    m3_joint j;
    m3_lines dh, dy, h, o, gate, dx, d_o, d_gate;
    float* sums[3];  // of weight, post_weight, scale (NULL: not asked for)
    float* parts;    // workspace: [3][norm_back_blocks][width]
    bool wide;
    hipStream_t stream;
};
hipError_t launch_norm_back(const NormBackArgs& a);

constexpr int kNormWidth = 8192, kNormForwardMost = 1024, kNormBackThreads = 512;
// Threads that share a row, 8 entries each, up to `most` of them (then 16).
// Rows without 16-byte accesses take a wave at least: their entries' addresses need registers.
inline int norm_row_threads(int width, bool wide, int most) {
    const int n = width <= 128 && wide ? 16 : width <= 512 ? 64 : width <= 1024 ? 128 : width <= 2048 ? 256 : width <= 4096 ? 512 : 1024;
    return n < most ? n : most;
}
// Workgroups that the backward pass deals the rows to: each keeps the sums of its rows and
// leaves one part of each, so there are no more of them than fill the chip.
inline int64_t norm_back_blocks(int64_t tokens, int width, bool wide) {
    const int64_t rows = kNormBackThreads / norm_row_threads(width, wide, kNormBackThreads);
    const int64_t n = (tokens + rows - 1) / rows;
    return n < 256 ? n : 256;
}

}  // namespace m3
