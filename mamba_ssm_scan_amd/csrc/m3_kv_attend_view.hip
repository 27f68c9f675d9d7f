// m3_kv_attend_view.hip -- the kernel for few rows (m3_kv_attend.hip) for calls with sinks or
// prefixes, in one pass over each sequence's keys: tiles go from the sinks' to the window's,
// and a sequence's first pages come from its group's table.
//
// Bound as the kernel without them: 128 sequences of 127 .. 16383 tokens under a window of 2048 with 64
// sinks (16 heads over 4 of 128, int8) 54 us, 4.7 TB/s of the keys seen; one sequence, window 1024,
// 9.6 us and its join's 3.8: latencies.
#include "m3_attend_rows.h"

namespace m3 {

hipError_t launch_rows_view(const AttendDev& d, m3_dtype io, hipStream_t s) { return launch_rows_form<kView>(d, io, s); }

}  // namespace m3
