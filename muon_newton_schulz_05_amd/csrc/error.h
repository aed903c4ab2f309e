// error.h -- the calling thread's last error message (muon_last_error).
#pragma once

namespace muon {

// Stores a printf-style message (empty: "") and returns code.
int set_error(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

}  // namespace muon
