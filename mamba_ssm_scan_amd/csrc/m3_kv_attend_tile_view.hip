// m3_kv_attend_tile_view.hip -- the kernel for many rows (m3_kv_attend_tile.hip) for calls with
// sinks or prefixes: kView as in m3_kv_attend_view.hip, kParts for the rows of a group over
// its prefix.
//
// Two prompts of 8192 under a window of 1024 with 16 sinks (16 heads over 4 of 128, e4m3): 224 us, 584
// TFLOP/s of the pairs seen, 644 of those computed. 2.1 us a tile, but 18 of them a
// workgroup only, beside 18 us that it takes at any window: 7.5 until the first scores (lengths, pages, codes,
// conversion, one after the other), the masks of the sinks' tile and of the window's ends, the first tile's
// maximum, the rows' way out. Workgroups of 4 waves and 128 rows, two a CU, hide that wait but convert
// each key twice as often: 233 us (window 512: 156 and 159).
// Eight questions of 256 behind 16384 tokens: 313 us with the join, 880 TFLOP/s.
#include "m3_attend_tile.h"

namespace m3 {

hipError_t launch_attend_tile_view(const AttendDev& d, m3_dtype io, hipStream_t s) {
    return d.form == kView ? launch_tile_form<kView>(d, io, s) : launch_tile_form<kParts>(d, io, s);
}

}  // namespace m3
