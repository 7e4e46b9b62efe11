// fo_error.hpp -- the per-thread message behind fo_last_error(), shared by the
// library's translation units (defined in fo_lib.hip).
#pragma once

namespace fo {
// record the message and return `code`
__attribute__((visibility("hidden"), format(printf, 2, 3))) int fail(int code, const char* fmt, ...);
__attribute__((visibility("hidden"))) void clear_error();
}  // namespace fo
