// m3_kv_attend_view.hip -- the kernel for few rows (m3_kv_attend.hip) for calls with sinks or
// prefixes, in one pass over each sequence's keys: tiles go from the sinks' to the window's,
// and a sequence's first pages come from its group's table.
#include "m3_attend_rows.h"

namespace m3 {

hipError_t launch_rows_view(const AttendDev& d, m3_dtype io, hipStream_t s) { return launch_rows_form<kView>(d, io, s); }

}  // namespace m3
