// m3_attn_stub_launch.cpp -- the attention layer's launchers replaced by stubs,
// for the host-only sanitizer build of its entry points (m3_attn_host.cpp). The
// argument checks return before any launch, so reaching a stub is a failure.
#include <cstdio>
#include <cstdlib>

#include "m3_attn_internal.h"

namespace m3 {
namespace {
[[noreturn]] void launched(const char* what) {
    std::fprintf(stderr, "host-only check build: %s reached a device launch\n", what);
    std::abort();
}
}  // namespace

hipError_t launch_rope(const RopeArgs&) { launched("launch_rope"); }
hipError_t launch_kv_append(const AppendArgs&) { launched("launch_kv_append"); }
hipError_t launch_kv_read(const ReadArgs&) { launched("launch_kv_read"); }
hipError_t launch_kv_attend(const AttendArgs&) { launched("launch_kv_attend"); }

}  // namespace m3
