// m3_host_checks.h -- what the entry points' argument checks share: ranges of bytes, and
// whether two sets of rows share any. Host code only.
#pragma once
#include <algorithm>
#include <cstdlib>

#include "../../include/m3_attn.h"
#include "m3_internal.h"

namespace m3 {
namespace {

inline size_t io_size(m3_dtype t) { return t == M3_BF16 ? 2 : 4; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline m3_status check_dtype(m3_dtype t) {
    if (t != M3_F32 && t != M3_BF16) return set_error(M3_EDTYPE, "unknown io dtype %d", (int)t);
    return M3_OK;
}

struct Range {
    const char* name;
    uintptr_t lo, hi;
};
inline bool overlaps(const Range& a, const Range& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
inline Range dense(const char* name, const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, p ? lo + bytes : lo};
}
// the bytes that rows cover, first to last
inline Range covered(const char* name, const m3_rows& r, int64_t tokens, int64_t heads, int64_t D, size_t es) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(r.p);
    if (!r.p || tokens == 0) return Range{name, lo, lo};
    return Range{name, lo, lo + size_t((tokens - 1) * r.token_stride + (heads - 1) * r.head_stride + D) * es};
}

// Whether two sets of rows share bytes. Parts of one fused projection interleave: by token
// (each part's heads together within a token stride; the common case, told by the parts'
// places in it) or by head as well ([token][head][part][D]). Rows of the same strides share
// bytes where some difference of their tokens and heads brings two of them closer than D.
inline bool rows_overlap(const m3_rows& a, int64_t a_heads, const m3_rows& b, int64_t b_heads, int64_t tokens, int64_t D,
                  size_t es) {
    if (!overlaps(covered("", a, tokens, a_heads, D, es), covered("", b, tokens, b_heads, D, es))) return false;
    const int64_t at = int64_t(reinterpret_cast<uintptr_t>(b.p)) - int64_t(reinterpret_cast<uintptr_t>(a.p));  // bytes
    if (tokens > 1 && a.token_stride != b.token_stride) return true;  // (not told apart: taken to overlap)
    const int64_t ts = a.token_stride * int64_t(es), row = D * int64_t(es);
    const int64_t ea = (a_heads - 1) * a.head_stride * int64_t(es) + row, eb = (b_heads - 1) * b.head_stride * int64_t(es) + row;
    if (tokens > 1 && ea <= ts && eb <= ts) {
        int64_t off = at % ts;
        if (off < 0) off += ts;
        if (off >= ea && off + eb <= ts) return false;
    }
    if (a_heads > 1 && b_heads > 1 && a.head_stride != b.head_stride) return true;
    const int64_t hs = (a_heads > 1 ? a : b).head_stride * int64_t(es);
    for (int64_t h = 1 - b_heads; h < a_heads; ++h) {  // a's head less b's
        const int64_t gap = at - h * hs;                // what the tokens' difference would have to make up
        int64_t t = tokens > 1 && ts > 0 ? gap / ts : 0;
        for (int64_t d = t - 1; d <= t + 1; ++d) {
            const int64_t n = std::max(1 - tokens, std::min(tokens - 1, d));
            if (std::abs(gap - n * ts) < row) return true;
        }
    }
    return false;
}

}  // namespace
}  // namespace m3
