// api_common.h -- what the translation units of the C ABI share: the calling
// thread's error text and its last kernel path.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/qlin.h"

namespace qlin {

// Sets the thread's error text and returns st.
qlin_status fail(qlin_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the error text.
qlin_status ok();
qlin_status device_status(hipError_t e, const char* what);
bool is_float_dtype(int d);
// Names the kernel path of the thread's last matmul-type call (a static string).
void record_path(const char* p);

}  // namespace qlin
