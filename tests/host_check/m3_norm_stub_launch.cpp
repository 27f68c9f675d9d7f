// m3_norm_stub_launch.cpp -- the joint's launchers replaced by stubs, for the
// host-only sanitizer build of its entry points (m3_norm_host.cpp). The
// argument checks return before any launch, so reaching a stub is a failure.
#include <cstdio>
#include <cstdlib>

#include "m3_norm_internal.h"

namespace m3 {
namespace {
[[noreturn]] void launched(const char* what) {
    std::fprintf(stderr, "host-only check build: %s reached a device launch\n", what);
    std::abort();
}
}  // namespace

hipError_t launch_norm(const NormArgs&) { launched("launch_norm"); }
hipError_t launch_norm_back(const NormBackArgs&) { launched("launch_norm_back"); }

}  // namespace m3
