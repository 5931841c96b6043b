// The library's last-error message, shared by its translation units.
#pragma once

#include "../../include/convfwd.h"

namespace convfwd {

// Records the message that conv_fwd_last_error returns on this thread and
// returns `st`.
conv_status_t fail(conv_status_t st, const char *fmt, ...) __attribute__((visibility("hidden"), format(printf, 2, 3)));

}  // namespace convfwd
