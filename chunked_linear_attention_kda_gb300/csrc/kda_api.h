// What the translation units that define C ABI entry points share: the thread's last error.
// Internal; not part of the C ABI.
#pragma once

#include <string>

#include "../../include/kda.h"

namespace kda {
kda_status api_fail(kda_status status, const std::string &why);  // sets kda_last_error, returns status
kda_status api_ok();                                             // clears it, returns KDA_OK
}  // namespace kda
