// The thread-local error text behind seed_last_error(), shared by the
// sources of the C ABI.
#pragma once

#include "../../include/seed.h"

namespace seed {

// Keeps `text` for seed_last_error() and returns `status`.
seed_status set_error(seed_status status, const char* text);

}  // namespace seed
