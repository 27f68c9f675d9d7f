// m3_kv_attend_tile_view.hip -- the kernel for many rows (m3_kv_attend_tile.hip) for calls with
// sinks or prefixes: kView as in m3_kv_attend_view.hip, kParts for the rows of a group over
// its prefix.
#include "m3_attend_tile.h"

namespace m3 {

hipError_t launch_attend_tile_view(const AttendDev& d, m3_dtype io, hipStream_t s) {
    return d.form == kView ? launch_tile_form<kView>(d, io, s) : launch_tile_form<kParts>(d, io, s);
}

}  // namespace m3
