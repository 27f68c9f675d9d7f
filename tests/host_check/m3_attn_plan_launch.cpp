// m3_attn_plan_launch.cpp -- the attention launcher replaced by one that notes the plan it was
// given, for tests of attend_plan's choices without a GPU.
#include "m3_attn_internal.h"

namespace m3 {
namespace {
AttendPlan noted;
}  // namespace

hipError_t launch_rope(const RopeArgs&) { return hipErrorUnknown; }
hipError_t launch_kv_append(const AppendArgs&) { return hipErrorUnknown; }
hipError_t launch_kv_read(const ReadArgs&) { return hipErrorUnknown; }
hipError_t launch_kv_attend(const AttendArgs& a) {
    noted = a.plan;
    return hipSuccess;
}

}  // namespace m3

// What the last attend call would have launched, as bits: the prefix apart, its launch the one for
// many rows, even shares.
extern "C" int m3_noted_plan() {
    const m3::AttendPlan& p = m3::noted;
    return (p.parts ? 1 : 0) | (p.parts && p.prefix.tile ? 2 : 0) | (p.items > 0 ? 4 : 0);
}
extern "C" int m3_noted_prefix_rows() { return m3::noted.prefix.rows; }
