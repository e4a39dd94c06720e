// Host-side helpers shared by the C-ABI translation units (no device code).
#pragma once

#include <cstdarg>
#include <cstddef>

namespace pa {

// Record a thread-local error message and return `code` (for `return fail(...)`).
int fail(int code, const char* fmt, ...);

// The current device's error word (device address) and SM count; PA_OK or a failure with its message.
int device_state(unsigned** error_word, int* num_sms);

// Clear the thread-local message (called on success paths that want it empty).
void clear_error();

}  // namespace pa
