// m3_norm_host.cpp -- the C entry points of the joint between two blocks
// (m3_norm.h): argument checks and dispatch. Host code only; every check runs
// before the first HIP call.
#include <cmath>

#include "m3_host_checks.h"
#include "m3_norm_internal.h"

namespace {

using m3::aligned;
using m3::covered;
using m3::dense;
using m3::overlaps;
using m3::Range;
using m3::set_error;

void clear_error() { set_error(M3_OK, "%s", ""); }

constexpr int64_t kMaxStride = int64_t(1) << 31;

m3_status check_joint(const m3_joint* j) {
    if (!j) return set_error(M3_EINVAL, "joint is NULL");
    for (const int32_t t : {j->stream_dtype, j->io_dtype})
        if (t != M3_F32 && t != M3_BF16) return set_error(M3_EDTYPE, "unknown dtype %d", t);
    if (j->stream_dtype == M3_BF16 && j->io_dtype == M3_F32)
        return set_error(M3_EUNSUPPORTED, "a bf16 stream with fp32 blocks");
    if (j->tokens < 0 || j->tokens > (int64_t(1) << 30))
        return set_error(M3_EINVAL, "tokens %lld out of range", (long long)j->tokens);
    if (j->width < 1) return set_error(M3_EINVAL, "width %d < 1", j->width);
    if (j->width > m3::kNormWidth) return set_error(M3_EUNSUPPORTED, "width %d above %d", j->width, m3::kNormWidth);
    if (j->gate_fn < M3_GATE_IDENTITY || j->gate_fn > M3_GATE_SIGMOID)
        return set_error(M3_EINVAL, "unknown gate function %d", j->gate_fn);
    if (!(j->eps >= 0.f) || !std::isfinite(j->eps)) return set_error(M3_EINVAL, "eps must be >= 0 and finite");
    if (!std::isfinite(j->factor)) return set_error(M3_EINVAL, "factor is not finite");
    const void* v[] = {j->scale, j->post_weight, j->weight};
    for (const void* p : v)
        if (!aligned(p, 4)) return set_error(M3_EALIGN, "scale, post_weight or weight is not 4-byte aligned");
    return M3_OK;
}

// Rows as one table of the checks has them.
struct Line {
    const char* name;
    const m3_lines* l;  // NULL: not given
    size_t es;
    bool out;
};
m3_rows as_rows(const Line& a) { return m3_rows{a.l->p, a.l->stride, 0}; }
Range range_of(const Line& a, const m3_joint& j) {
    if (!a.l) return Range{a.name, 0, 0};
    return covered(a.name, as_rows(a), j.tokens, 1, j.width, a.es);
}
m3_status check_line(const Line& a, const m3_joint& j) {
    if (!a.l) return M3_OK;
    if (!a.l->p && j.tokens > 0) return set_error(M3_EINVAL, "%s is NULL", a.name);
    if (!aligned(a.l->p, a.es)) return set_error(M3_EALIGN, "%s is not aligned to its entries", a.name);
    if (a.l->stride < 0 || a.l->stride > kMaxStride)
        return set_error(M3_EINVAL, "%s: the stride is negative or above 2^31", a.name);
    if (a.out && j.tokens > 1 && a.l->stride < j.width) return set_error(M3_EINVAL, "%s: rows overlap (stride)", a.name);
    return M3_OK;
}
bool same(const Line& a, const Line& b, const m3_joint& j) {
    return a.l && b.l && a.l->p == b.l->p && a.es == b.es && (j.tokens <= 1 || a.l->stride == b.l->stride);
}
bool share(const Line& a, const Line& b, const m3_joint& j) {
    if (!a.l || !b.l || !overlaps(range_of(a, j), range_of(b, j))) return false;
    return a.es != b.es || m3::rows_overlap(as_rows(a), 1, as_rows(b), 1, j.tokens, j.width, a.es);
}
bool wide_line(const Line& a, const m3_joint& j) {
    return !a.l || (aligned(a.l->p, 16) && (j.tokens <= 1 || a.l->stride * a.es % 16 == 0));
}
bool wide_vector(const void* p) { return aligned(p, 16); }
m3_lines of(const m3_lines* l) { return l ? *l : m3_lines{nullptr, 0}; }

// Outputs apart from inputs and each other. in_place[i]: the input that lines[i] may be, or -1.
template <int N>
m3_status check_lines(const Line (&lines)[N], const int (&in_place)[N], const m3_joint& j) {
    for (const Line& a : lines) {
        const m3_status s = check_line(a, j);
        if (s != M3_OK) return s;
    }
    const Range vectors[] = {dense("scale", j.scale, size_t(j.width) * 4),
                             dense("post_weight", j.post_weight, size_t(j.width) * 4),
                             dense("weight", j.weight, size_t(j.width) * 4)};
    for (int a = 0; a < N; ++a) {
        if (!lines[a].out || !lines[a].l) continue;
        for (int b = 0; b < N; ++b) {
            if (a == b || (lines[b].out && b < a)) continue;
            if (in_place[a] == b && same(lines[a], lines[b], j)) continue;
            if (share(lines[a], lines[b], j)) return set_error(M3_EINVAL, "%s overlaps %s", lines[a].name, lines[b].name);
        }
        for (const Range& v : vectors)
            if (overlaps(range_of(lines[a], j), v)) return set_error(M3_EINVAL, "%s overlaps %s", lines[a].name, v.name);
    }
    return M3_OK;
}

}  // namespace

extern "C" {

m3_status m3_residual_norm(const m3_joint* joint, const m3_lines* x, const m3_lines* o, const m3_lines* gate,
                           const m3_lines* h, const m3_lines* y, void* stream) {
    clear_error();
    m3_status s = check_joint(joint);
    if (s != M3_OK) return s;
    const m3_joint& j = *joint;
    if (!x) return set_error(M3_EINVAL, "x is NULL");
    if (!o && (gate || h)) return set_error(M3_EINVAL, "gate or h without o");
    if (o && !h) return set_error(M3_EINVAL, "h is NULL");
    if ((y == nullptr) != (j.weight == nullptr)) return set_error(M3_EINVAL, "y and weight must be given together");
    if (!o && !y) return set_error(M3_EINVAL, "neither o nor weight is given");
    const size_t xs = m3::io_size(m3_dtype(j.stream_dtype)), os = m3::io_size(m3_dtype(j.io_dtype));
    const Line lines[] = {{"x", x, xs, false}, {"o", o, os, false}, {"gate", gate, os, false}, {"h", h, xs, true},
                          {"y", y, os, true}};
    const int in_place[] = {-1, -1, -1, 0, o ? 1 : 0};
    if ((s = check_lines(lines, in_place, j)) != M3_OK) return s;
    if (j.tokens == 0) return M3_OK;
    bool wide = j.width % 8 == 0 && wide_vector(j.scale) && wide_vector(j.post_weight) && wide_vector(j.weight);
    for (const Line& a : lines) wide = wide && wide_line(a, j);
    m3::NormArgs a{j, *x, of(o), of(gate), of(h), of(y), wide, reinterpret_cast<hipStream_t>(stream)};
    const hipError_t e = m3::launch_norm(a);
    if (e != hipSuccess) return set_error(M3_EHIP, "residual norm launch failed: %s", hipGetErrorString(e));
    return M3_OK;
}

size_t m3_residual_norm_backward_workspace_size(const m3_joint* joint, int32_t sums) {
    clear_error();
    if (check_joint(joint) != M3_OK || !sums) return 0;
    // (without 16-byte accesses there may be more parts, never fewer)
    return size_t(3) * size_t(m3::norm_back_blocks(joint->tokens, joint->width, false)) * size_t(joint->width) * 4;
}

m3_status m3_residual_norm_backward(const m3_joint* joint, const m3_lines* dh, const m3_lines* dy, const m3_lines* h,
                                    const m3_lines* o, const m3_lines* gate, const m3_lines* dx, const m3_lines* d_o,
                                    const m3_lines* d_gate, float* d_weight, float* d_post_weight, float* d_scale,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    m3_status s = check_joint(joint);
    if (s != M3_OK) return s;
    const m3_joint& j = *joint;
    if ((dy == nullptr) != (j.weight == nullptr)) return set_error(M3_EINVAL, "dy and weight must be given together");
    if (!dh && !dy) return set_error(M3_EINVAL, "neither dh nor dy is given");
    if (dy && !h) return set_error(M3_EINVAL, "h is NULL");
    if (!o && (gate || d_o || d_gate || d_post_weight || d_scale))
        return set_error(M3_EINVAL, "gate or a gradient of the branch without o");
    if (d_gate && !gate) return set_error(M3_EINVAL, "d_gate without gate");
    if (d_weight && !j.weight) return set_error(M3_EINVAL, "d_weight without weight");
    if (d_post_weight && !j.post_weight) return set_error(M3_EINVAL, "d_post_weight without post_weight");
    if (d_scale && !j.scale) return set_error(M3_EINVAL, "d_scale without scale");
    if (!dx && !d_o && !d_gate && !d_weight && !d_post_weight && !d_scale)
        return set_error(M3_EINVAL, "no gradient is asked for");
    const size_t xs = m3::io_size(m3_dtype(j.stream_dtype)), os = m3::io_size(m3_dtype(j.io_dtype));
    const Line lines[] = {{"dh", dh, xs, false}, {"dy", dy, os, false},  {"h", h, xs, false},  {"o", o, os, false},
                          {"gate", gate, os, false}, {"dx", dx, xs, true}, {"d_o", d_o, os, true}, {"d_gate", d_gate, os, true}};
    const int in_place[] = {-1, -1, -1, -1, -1, 0, -1, -1};
    if ((s = check_lines(lines, in_place, j)) != M3_OK) return s;
    const bool sums = d_weight || d_post_weight || d_scale;
    const size_t need = m3_residual_norm_backward_workspace_size(joint, sums);
    const size_t vec = size_t(j.width) * 4;
    const Range outs[] = {dense("d_weight", d_weight, vec), dense("d_post_weight", d_post_weight, vec),
                          dense("d_scale", d_scale, vec), dense("workspace", workspace, workspace_bytes)};
    const Range vectors[] = {dense("scale", j.scale, vec), dense("post_weight", j.post_weight, vec), dense("weight", j.weight, vec)};
    for (int a = 0; a < 4; ++a) {
        for (const Line& l : lines)
            if (overlaps(outs[a], range_of(l, j))) return set_error(M3_EINVAL, "%s overlaps %s", outs[a].name, l.name);
        for (const Range& v : vectors)
            if (overlaps(outs[a], v)) return set_error(M3_EINVAL, "%s overlaps %s", outs[a].name, v.name);
        for (int b = a + 1; b < 4; ++b)
            if (overlaps(outs[a], outs[b])) return set_error(M3_EINVAL, "%s overlaps %s", outs[a].name, outs[b].name);
    }
    float* const sum[] = {d_weight, d_post_weight, d_scale};
    for (const float* p : sum)
        if (!aligned(p, 4)) return set_error(M3_EALIGN, "d_weight, d_post_weight or d_scale is not 4-byte aligned");
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return set_error(M3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
        if (!aligned(workspace, 16)) return set_error(M3_EALIGN, "workspace is not 16-byte aligned");
    }
    if (j.tokens == 0 && !sums) return M3_OK;
    bool wide = j.width % 8 == 0 && wide_vector(j.scale) && wide_vector(j.post_weight) && wide_vector(j.weight);
    for (const Line& a : lines) wide = wide && wide_line(a, j);
    m3::NormBackArgs a{j, of(dh), of(dy), of(h), of(o), of(gate), of(dx), of(d_o), of(d_gate),
                       {d_weight, d_post_weight, d_scale}, static_cast<float*>(workspace), wide,
                       reinterpret_cast<hipStream_t>(stream)};
    const hipError_t e = m3::launch_norm_back(a);
    if (e != hipSuccess) return set_error(M3_EHIP, "residual norm backward launch failed: %s", hipGetErrorString(e));
    return M3_OK;
}

}  // extern "C"
